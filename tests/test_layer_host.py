"""The operators around the attention on the host (no GPU): argument checks with fake,
never-dereferenced pointers, the position packer, and the binding's own refusals."""
import ctypes

import numpy as np
import pytest

import video_diffusion_attention_b200 as T
from video_diffusion_attention_b200 import _binding as B
from video_diffusion_attention_b200 import build as libbuild

OK, NULL, SHAPE, DTYPE, HEAD_DIM, PARAM, ALIGN = 0, -1, -2, -3, -4, -5, -6
SEGMENT, CAPACITY, TOO_LARGE = -7, -8, -11
FAKE, FAKE2, FAKE3, FAKE4, FAKE5 = (0x7f0000000000 + i * 0x1000000000 for i in range(1, 6))


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return B.load_library()


def view(ptr=FAKE, dtype=B.TARA_BF16, shape=(1, 2, 300, 128), strides=None):
    v = B.TaraView()
    v.ptr, v.dtype = ptr, dtype
    v.B, v.H, v.N, v.D = shape
    if strides is None:
        strides = (shape[1] * shape[2] * shape[3], shape[2] * shape[3], shape[3])
    v.stride_b, v.stride_h, v.stride_n = strides
    return v


def stream_view(ptr, N, C, dtype=B.TARA_BF16, nb=1):
    return view(ptr, dtype, (nb, 1, N, C), (N * C, 0, C))


def norm_rope(**kw):
    p = B.TaraNormRope()
    p.norm, p.eps, p.table, p.rot_dim = 1, 1e-6, FAKE5, 128
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def ref(x):
    return ctypes.byref(x) if x is not None else None


# ---------------------------------------------------------------------------------------
# rope_table
# ---------------------------------------------------------------------------------------
def rope(dims, thetas):
    r = B.TaraRope()
    r.n_axes = len(dims)
    for i, (d, t) in enumerate(zip(dims, thetas)):
        r.dim[i], r.theta[i] = d, t
    return r


@pytest.mark.parametrize("dims,thetas,want", [
    ((), (), PARAM),
    ((16, 56, 55), (1e4,) * 3, SHAPE),          # odd axis
    ((0, 64), (1e4,) * 2, SHAPE),
    ((128, 130), (1e4,) * 2, SHAPE),            # more than 256 columns
    ((2, 4), (1e4,) * 2, SHAPE),                # not a multiple of 4
    ((64,), (0.0,), PARAM),
    ((64,), (float("nan"),), PARAM),
    ((64,), (float("inf"),), PARAM),
])
def test_rope_table_refuses(lib, dims, thetas, want):
    assert lib.tara_rope_table(FAKE, 10, ref(rope(dims, thetas)), FAKE2, None) == want


def test_rope_table_refuses_pointers_and_sizes(lib):
    r = rope((64,), (1e4,))
    assert lib.tara_rope_table(None, 10, ref(r), FAKE, None) == NULL
    assert lib.tara_rope_table(FAKE, 10, None, FAKE, None) == NULL
    assert lib.tara_rope_table(FAKE, 10, ref(r), None, None) == NULL
    assert lib.tara_rope_table(FAKE, 0, ref(r), FAKE2, None) == SHAPE
    assert lib.tara_rope_table(FAKE + 2, 10, ref(r), FAKE2, None) == ALIGN
    assert lib.tara_rope_table(FAKE, 10, ref(r), FAKE2 + 8, None) == ALIGN
    assert lib.tara_rope_table(FAKE, 1 << 41, ref(r), FAKE2, None) == TOO_LARGE
    r.n_axes = 5
    assert lib.tara_rope_table(FAKE, 10, ref(r), FAKE2, None) == PARAM


# ---------------------------------------------------------------------------------------
# qk_norm_rope
# ---------------------------------------------------------------------------------------
def call_qk(lib, q=None, k=None, p=None, qo=None, ko=None):
    q = q or view(FAKE)
    k = k or view(FAKE2)
    qo = qo or view(FAKE3)
    ko = ko or view(FAKE4)
    return lib.tara_qk_norm_rope(ref(q), ref(k), ref(p or norm_rope()), ref(qo), ref(ko), None)


def test_qk_norm_rope_refuses_null(lib):
    v, p = view(), norm_rope()
    f = lib.tara_qk_norm_rope
    assert f(None, ref(v), ref(p), ref(v), ref(v), None) == NULL
    assert f(ref(v), ref(v), None, ref(v), ref(v), None) == NULL
    assert f(ref(v), None, ref(p), None, None, None) == NULL
    assert f(ref(v), None, ref(p), ref(v), ref(v), None) == NULL      # k_out without k
    assert f(ref(v), ref(v), ref(p), ref(v), None, None) == NULL      # k without k_out
    assert call_qk(lib, q=view(None)) == NULL


@pytest.mark.parametrize("kw,want", [
    (dict(shape=(0, 2, 300, 128)), SHAPE), (dict(shape=(1, 2, 0, 128)), SHAPE),
    (dict(shape=(1, 2, 301, 128)), SHAPE),                       # unlike the others
    (dict(dtype=B.TARA_FP16), DTYPE), (dict(dtype=7), DTYPE),
    (dict(ptr=FAKE2 + 8), ALIGN),
    (dict(strides=(0, 300 * 128 + 4, 128)), ALIGN),
    (dict(strides=(0, -128, 128)), PARAM),
    (dict(strides=(0, 1 << 39, 128)), TOO_LARGE),
])
def test_qk_norm_rope_refuses_views(lib, kw, want):
    kw = dict(kw)
    ptr = kw.pop("ptr", FAKE2)
    assert call_qk(lib, k=view(ptr, **kw)) == want


@pytest.mark.parametrize("shape", [(1, 2, 300, 132), (1, 2, 300, 264), (1, 2, 300, 4)])
def test_qk_norm_rope_refuses_head_dims(lib, shape):
    strides = (1 << 20, 1 << 19, 512)
    vs = [view(p, shape=shape, strides=strides) for p in (FAKE, FAKE2, FAKE3, FAKE4)]
    assert call_qk(lib, vs[0], vs[1], norm_rope(rot_dim=8), vs[2], vs[3]) == HEAD_DIM


@pytest.mark.parametrize("strides", [(0, 0, 128), (0, 300 * 128, 64), (0, 64, 128)])
def test_outputs_may_not_overlap_themselves(lib, strides):
    # two heads on one another, rows on one another, heads inside a row
    assert call_qk(lib, qo=view(FAKE3, strides=strides)) == PARAM
    # (two overlapping inputs, such as an expanded head, are fine: nothing else is refused)


@pytest.mark.parametrize("kw,want", [
    (dict(norm=0, table=None), PARAM), (dict(norm=2), PARAM),
    (dict(eps=-1.0), PARAM), (dict(eps=float("nan")), PARAM), (dict(eps=float("inf")), PARAM),
    (dict(rot_dim=0), PARAM), (dict(rot_dim=136), PARAM), (dict(rot_dim=4), PARAM),
    (dict(rot_dim=8, pairing=1), PARAM), (dict(pairing=2), PARAM), (dict(pairing=-1), PARAM),
    (dict(table=FAKE5 + 4), ALIGN), (dict(table_batch_stride=300 * 128 - 4), PARAM),
    (dict(table_batch_stride=300 * 128 + 2), ALIGN), (dict(table_batch_stride=-4), PARAM),
    (dict(q_weight=FAKE + 2), ALIGN), (dict(k_weight=FAKE + 8), ALIGN),
    (dict(weight_head_stride=64), PARAM), (dict(weight_head_stride=-128), PARAM),
    (dict(weight_head_stride=132), ALIGN),
])
def test_qk_norm_rope_refuses_parameters(lib, kw, want):
    assert call_qk(lib, p=norm_rope(**kw)) == want


def test_qk_norm_rope_refuses_shared_buffers(lib):
    assert call_qk(lib, qo=view(FAKE2)) == PARAM                      # q_out over k
    assert call_qk(lib, ko=view(FAKE)) == PARAM
    assert call_qk(lib, ko=view(FAKE3)) == PARAM                      # both outputs in one place
    # an output in its input's place must have its layout
    assert call_qk(lib, qo=view(FAKE, strides=(0, 128, 256))) == PARAM


def test_qk_norm_rope_refuses_too_many_heads(lib):
    vs = [view(p, shape=(1, 40000, 1, 8)) for p in (FAKE, FAKE2, FAKE3, FAKE4)]
    assert call_qk(lib, vs[0], vs[1], norm_rope(rot_dim=8), vs[2], vs[3]) == TOO_LARGE


# ---------------------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------------------
def epilogue(**kw):
    e = B.TaraEpilogue()
    keep = kw.pop("residual", None)
    if keep is not None:
        e.residual = ctypes.pointer(keep)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def call_linear(lib, x=None, w=FAKE2, e=None, y=None):
    x = x or stream_view(FAKE, 300, 256)
    y = y or stream_view(FAKE3, 300, 512)
    return lib.tara_linear(ref(x), w, ref(e), ref(y), None)


def test_linear_refuses_null(lib):
    v = stream_view(FAKE, 300, 256)
    assert lib.tara_linear(None, FAKE2, None, ref(v), None) == NULL
    assert lib.tara_linear(ref(v), None, None, ref(v), None) == NULL
    assert lib.tara_linear(ref(v), FAKE2, None, None, None) == NULL


@pytest.mark.parametrize("x,want", [
    (stream_view(FAKE, 0, 256), SHAPE), (stream_view(FAKE, 301, 256), SHAPE),
    (view(FAKE, shape=(1, 1, 300, 252), strides=(0, 0, 256)), SHAPE),  # not a multiple of 8
    (view(FAKE, shape=(1, 4, 300, 72)), SHAPE),                        # heads not of 64 columns
    (stream_view(FAKE, 300, 256, B.TARA_FP16), DTYPE),
    (stream_view(FAKE + 2, 300, 256), ALIGN),
    (view(FAKE, shape=(1, 1, 300, 256), strides=(0, 0, 260)), ALIGN),
    (stream_view(FAKE3, 300, 256), PARAM),                             # y over x
    (view(FAKE, shape=(1, 1, 300, 256), strides=(0, 0, 0)), PARAM),    # one row, expanded
    (view(FAKE, shape=(1, 2, 300, 128), strides=(0, 0, 128)), PARAM),  # one head, expanded
])
def test_linear_refuses_inputs(lib, x, want):
    assert call_linear(lib, x=x) == want


@pytest.mark.parametrize("kw,want", [
    (dict(act=4), PARAM), (dict(act=-1), PARAM), (dict(bias=FAKE + 2), ALIGN),
    (dict(gate=FAKE + 8), ALIGN), (dict(gate=FAKE, gate_stride=256), PARAM),
    (dict(gate=FAKE, gate_stride=-512), PARAM), (dict(gate=FAKE, gate_stride=516), ALIGN),
    (dict(residual=stream_view(FAKE4, 300, 256)), SHAPE),
    (dict(residual=stream_view(FAKE4, 299, 512)), SHAPE),
    (dict(residual=stream_view(FAKE4, 300, 512, B.TARA_FP16)), DTYPE),
    (dict(residual=stream_view(FAKE4 + 4, 300, 512)), ALIGN),
    (dict(residual=view(FAKE3, shape=(1, 4, 300, 128))), PARAM),       # in y's place, another layout
])
def test_linear_refuses_epilogues(lib, kw, want):
    assert call_linear(lib, e=epilogue(**kw)) == want


def test_linear_refuses_weights_and_outputs(lib):
    assert call_linear(lib, w=FAKE2 + 8) == ALIGN
    assert call_linear(lib, w=FAKE3) == PARAM
    assert call_linear(lib, y=view(FAKE3, shape=(1, 1, 300, 512), strides=(0, 0, 0))) == PARAM
    assert call_linear(lib, y=view(FAKE3, shape=(1, 8, 300, 68))) == ALIGN
    f = B.TARA_FP32
    assert call_linear(lib, stream_view(FAKE, 300, 255, f), FAKE2 + 2, None,
                       stream_view(FAKE3, 300, 511, f)) == ALIGN


# ---------------------------------------------------------------------------------------
# qkv_project
# ---------------------------------------------------------------------------------------
def call_qkv(lib, x=None, w=FAKE2, bias=None, p=None, q=None, k=None, v=None):
    x = x or stream_view(FAKE, 300, 256)
    q, k, v = (o or view(a) for o, a in ((q, FAKE3), (k, FAKE4), (v, FAKE5 + (1 << 34))))
    return lib.tara_qkv_project(ref(x), w, bias, ref(p), ref(q), ref(k), ref(v), None)


def test_qkv_project_refuses(lib):
    assert lib.tara_qkv_project(None, FAKE, None, None, None, None, None, None) == NULL
    assert call_qkv(lib, w=None) == NULL
    assert call_qkv(lib, x=stream_view(FAKE, 299, 256)) == SHAPE
    assert call_qkv(lib, v=view(FAKE5, shape=(1, 2, 300, 64))) == SHAPE
    assert call_qkv(lib, k=view(FAKE4, dtype=B.TARA_FP16)) == DTYPE
    assert call_qkv(lib, k=view(FAKE3)) == PARAM
    assert call_qkv(lib, q=view(FAKE)) == PARAM
    assert call_qkv(lib, bias=FAKE5 + 2) == ALIGN
    assert call_qkv(lib, v=view(FAKE5, strides=(0, 0, 128))) == PARAM
    assert call_qkv(lib, p=norm_rope(rot_dim=136)) == PARAM
    outs = [view(a, shape=(1, 2, 300, 96)) for a in (FAKE3, FAKE4, FAKE5)]
    assert call_qkv(lib, None, FAKE2, None, None, *outs) == HEAD_DIM
    f = B.TARA_FP32
    outs = [view(a, f, (1, 2, 300, 20)) for a in (FAKE3, FAKE4, FAKE5)]
    assert call_qkv(lib, stream_view(FAKE, 300, 256, f), FAKE2, None, None, *outs) == HEAD_DIM


@pytest.mark.parametrize("K", [2 ** 31 - 1, 2 ** 31 - 8, 2 ** 31 - 64, 2 ** 31 - 248])
@pytest.mark.parametrize("dtype", [B.TARA_FP32, B.TARA_BF16])
@pytest.mark.parametrize("N", [1, 8, 9, 300])
def test_input_columns_leave_room_for_a_step_of_the_kernels(lib, N, dtype, K):
    # the kernels count input columns in int and step past the last one by less than 256; with
    # fp32 one row may stand for all tokens (8 GB), so that such a call is possible
    if dtype == B.TARA_BF16:
        K -= K % 8
    x = view(FAKE, dtype, (1, 1, N, K), (0, 0, 0 if dtype == B.TARA_FP32 else 1 << 31))
    assert call_linear(lib, x, FAKE2, None, view(FAKE3, dtype, (1, 1, N, 8))) == TOO_LARGE
    outs = [view(a, dtype, (1, 1, N, 64)) for a in (FAKE3, FAKE4, FAKE5)]
    assert call_qkv(lib, x, FAKE2, None, None, *outs) == TOO_LARGE


def test_input_columns_count_over_all_heads(lib):
    heads = view(FAKE, B.TARA_BF16, (1, (1 << 25) - 1, 1, 64), (0, 64, 0))
    assert call_linear(lib, heads, FAKE2, None, stream_view(FAKE3, 1, 8)) == TOO_LARGE


# ---------------------------------------------------------------------------------------
# positions
# ---------------------------------------------------------------------------------------
def test_positions_of_a_packed_shot():
    dt = 4.0 / 24.0
    grids = [T.TokenGrid(frames=3), T.TokenGrid(frames=2, rows=2, cols=3, origin=(3.0, -0.5, 10.0),
                                                frame_step=(dt, 0.0, 0.0)),
             T.TokenGrid(1, origin=(7.0, 1.0, 2.0))]
    pos = T.pack_token_positions(grids)
    want = [(i, 0, 0) for i in range(3)]
    want += [(3.0 + f * dt, -0.5 + r, 10.0 + c) for f in range(2) for r in range(2)
             for c in range(3)]
    want += [(7.0, 1.0, 2.0)]
    assert pos.dtype == np.float32 and pos.shape == (16, 3)
    assert np.array_equal(pos, np.array(want, np.float64).astype(np.float32))


def test_positions_with_other_axis_counts():
    # one axis, and four with diagonal text (every axis advances)
    assert np.array_equal(T.pack_token_positions([T.TokenGrid(5)], 1)[:, 0], np.arange(5))
    diag = T.TokenGrid(4, origin=(1,) * 4, frame_step=(1,) * 4, row_step=(0,) * 4, col_step=(0,) * 4)
    assert np.array_equal(T.pack_token_positions([diag], 4), np.arange(1, 5)[:, None] * np.ones(4))
    assert T.pack_token_positions([]).shape == (0, 3)


@pytest.mark.parametrize("grid", [T.TokenGrid(0), T.TokenGrid(1, -1), T.TokenGrid(1, 1, 0),
                                  T.TokenGrid(1, origin=(float("nan"), 0, 0)),
                                  T.TokenGrid(1, col_step=(0, float("inf"), 0))])
def test_positions_refuse_bad_grids(grid):
    with pytest.raises(B.TaraError) as e:
        T.pack_token_positions([T.TokenGrid(2), grid])
    assert e.value.code == SEGMENT


def test_positions_refuse_lengths_and_axes(lib):
    arr = (B.TaraGrid * 1)()
    arr[0].frames, arr[0].rows, arr[0].cols = 2, 3, 4
    buf = np.full(3 * 24, 7.0, np.float32)
    f = lib.tara_pack_token_positions
    for N in (-1, 0, 23, 25):
        assert f(arr, 1, 3, buf.ctypes.data, N) == CAPACITY
    assert f(arr, 1, 0, buf.ctypes.data, 24) == PARAM
    assert f(arr, 1, 5, buf.ctypes.data, 24) == PARAM
    assert f(arr, -1, 3, buf.ctypes.data, 24) == SEGMENT
    assert f(None, 1, 3, buf.ctypes.data, 24) == NULL
    assert f(arr, 1, 3, None, 24) == NULL
    arr[0].frames = arr[0].rows = arr[0].cols = 2 ** 31 - 1          # a product past 64 bits
    assert f(arr, 1, 3, buf.ctypes.data, 24) == CAPACITY
    assert np.all(buf == 7.0)


# ---------------------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------------------
def test_binding_refuses_host_tensors():
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for f in (lambda: T.linear(x, x), lambda: T.qkv_project(x, x, 1), lambda: T.rope_table(x, [8]),
              lambda: T.qk_norm_rope(x[None, None])):
        with pytest.raises(ValueError):
            f()


class NoCalls:
    """A library of which nothing may be called."""

    def __getattr__(self, name):
        raise AssertionError("%s was called" % name)


@pytest.mark.parametrize("shape", [
    (2, 4, 30, 64),      # more heads than w has rows
    (2, 1, 30, 64),      # fewer
    (2, 2, 30, 128),     # longer heads
    (2, 4, 30, 32),      # the same columns in other heads
    (2, 1, 30, 128),     # the same columns in one head
    (2, 30, 128),        # token-major
    (2, 30, 64),         # token-major, one head
    (2, 2, 31, 64),      # another number of tokens
    (1, 2, 30, 64),      # one branch
])
@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_binding_refuses_outputs_unlike_the_projection(monkeypatch, dtype, which, shape):
    # The library sees w as a pointer and takes its rows from the outputs: outputs of other sizes
    # would read behind w, bias and weights.  Refused before any library call (host tensors here).
    import torch
    from video_diffusion_attention_b200 import _layer
    monkeypatch.setattr(_layer, "_elsewhere", lambda t, stream: None)
    monkeypatch.setattr(_layer, "_current_stream", lambda t: 0)
    monkeypatch.setattr(_layer, "load_library", NoCalls)
    dt = getattr(torch, dtype)
    heads, D, K = 2, 64, 96
    x, w = torch.zeros(2, 30, K, dtype=dt), torch.zeros(3 * heads * D, K, dtype=dt)
    out = [torch.zeros(2, heads, 30, D, dtype=dt) for _ in range(3)]
    out[which] = torch.zeros(shape, dtype=dt)
    with pytest.raises(ValueError):
        T.qkv_project(x, w, heads, bias=torch.zeros(3 * heads * D, dtype=dt),
                      q_weight=torch.ones(heads, D, dtype=dt), out=out)
    with pytest.raises(ValueError):
        T.qkv_project(x, w, heads, out=[torch.zeros(shape, dtype=dt)] * 3)
    with pytest.raises(ValueError):
        T.qkv_project(x, w, heads, out=out[:2])


def test_struct_sizes_match_the_header(tmp_path):
    # the ctypes layouts against the C compiler's
    import os
    import subprocess
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    names = {"tara_view": B.TaraView, "tara_rope": B.TaraRope, "tara_norm_rope": B.TaraNormRope,
             "tara_epilogue": B.TaraEpilogue, "tara_grid": B.TaraGrid}
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "tara_attn.h"\nint main(void) {\n'
    for n, c in names.items():
        src += 'printf("%%zu\\n", sizeof(%s));\n' % n
        for f in c._fields_:
            src += 'printf("%%zu\\n", offsetof(%s, %s));\n' % (n, f[0])
    (tmp_path / "s.c").write_text(src + "return 0; }\n")
    subprocess.check_call(["gcc", "-std=c99", "-I", inc, str(tmp_path / "s.c"), "-o", str(tmp_path / "s")])
    got = [int(v) for v in subprocess.check_output([str(tmp_path / "s")]).split()]
    want = []
    for c in names.values():
        want += [ctypes.sizeof(c)] + [getattr(c, f[0]).offset for f in c._fields_]
    assert got == want
