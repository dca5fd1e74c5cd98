"""The operators around the attention on the GPU against their fp64 definitions (oracle/layer.py).

Tolerance of every element: the fp32 bound that comes with the definition, plus half a unit of
the output's type (relative to value and bound), plus half the type's smallest subnormal.
"""
import numpy as np
import pytest
import torch

import video_diffusion_attention_b200 as T
from oracle import layer as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}


def np64(t):
    return t.detach().double().cpu().numpy()


def rand(shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float32) * scale + shift
    return x.to(DT[dtype]).cuda()


def close(got, value, bound, dtype):
    got = np64(got).reshape(value.shape)
    half = torch.finfo(DT[dtype]).eps / 2
    tol = bound + half * (np.abs(value) + bound) + TINY[dtype]
    assert np.all(np.isfinite(got))
    worst = np.max((np.abs(got - value) - tol))
    assert worst <= 0, "beyond tolerance by %g (tolerance up to %g)" % (worst, tol.max())


def positions(N, axes, seed, far=0.0):
    g = np.random.Generator(np.random.PCG64(seed))
    p = g.uniform(-20.0, 50.0, size=(N, axes)) + far
    return torch.from_numpy(p.astype(np.float32)).cuda()


def table_for(N, dims, seed, B=0):
    """A random (cos, sin) table [N or B,N][R/2][2]."""
    g = np.random.Generator(np.random.PCG64(seed))
    a = g.uniform(-np.pi, np.pi, size=((B,) if B else ()) + (N, sum(dims) // 2))
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)).cuda()


# ---------------------------------------------------------------------------------------
# rope_table
# ---------------------------------------------------------------------------------------
@pytest.mark.parametrize("N,dims,theta,far", [
    (1, (64,), 10000.0, 0.0), (3, (2, 2), 10.0, 0.0), (257, (16, 56, 56), 10000.0, 0.0),
    (1000, (44, 42, 42), 256.0, 1e6), (33, (64, 64, 64, 64), 1e6, -3e8),
    (129, (128, 128), (500.0, 2e5), 2.0 ** 30), (5, (2, 120, 6), 1.0, 7e4),
])
def test_rope_table(N, dims, theta, far):
    pos = positions(N, len(dims), N, far)
    thetas = theta if isinstance(theta, tuple) else (theta,) * len(dims)
    got = np64(T.rope_table(pos, dims, theta))
    a = ref.angles(pos.cpu().numpy(), dims, thetas)
    # the fp64 angle carries a few units of 2^-53 relative; what is left of it after the whole
    # quarter turns is rounded to fp32 (at most pi/4 * 2^-24), then cos or sin to 2 units
    tol = np.abs(a)[..., None] * 2.0 ** -50 + 2.0 ** -24 + 2 * 2.0 ** -23 * np.stack(
        [np.abs(np.cos(a)), np.abs(np.sin(a))], -1)
    want = np.stack([np.cos(a), np.sin(a)], -1)
    assert got.shape == want.shape
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want))


@pytest.mark.parametrize("far", [0.0, 5e4, 2.0 ** 30])
def test_rope_table_error_bound(far):
    # The bound the header states: 1e-7 beside the error of the fp64 angle (2^-50 relative, the
    # definition's own included).  Counted: the remainder rounded to fp32 below pi/4, 2^-25; the
    # last fma of a series below 1, 2^-25; its inner terms below 2^-25.5; the series, 2^-29.
    pos = positions(20000, 3, 77, far)
    got = np64(T.rope_table(pos, (16, 56, 56)))
    a = ref.angles(pos.cpu().numpy(), (16, 56, 56), (1e4,) * 3)
    err = np.abs(got - np.stack([np.cos(a), np.sin(a)], -1))
    assert np.all(err <= 1e-7 + np.abs(a)[..., None] * 2.0 ** -50), err.max()


def test_rope_table_of_packed_positions_and_branches():
    grids = [T.TokenGrid(frames=7), T.TokenGrid(3, 4, 5, origin=(7.0, 0.0, 0.0),
                                                frame_step=(4 / 24, 0, 0))]
    pos = torch.from_numpy(T.pack_token_positions(grids)).cuda()
    one = T.rope_table(pos, (8, 12, 12))
    both = T.rope_table(torch.stack([pos, pos + 1.0]), (8, 12, 12))
    assert both.shape == (2, 67, 16, 2) and torch.equal(both[0], one)
    assert torch.equal(one[0, :, 0], torch.ones(16, device="cuda"))       # position 0: no turn
    out = torch.full((68, 16, 2), 7.0, device="cuda")
    T.rope_table(pos, (8, 12, 12), out=out[:67])
    assert torch.equal(out[:67], one) and bool((out[67] == 7.0).all())


# ---------------------------------------------------------------------------------------
# qk_norm_rope
# ---------------------------------------------------------------------------------------
def layout(kind, B, H, N, D, dtype, seed):
    """Q or K of one layout, as a [B][H][N][D] view."""
    if kind == "heads":
        return rand((B, H, N, D), dtype, seed, 1.5)
    if kind == "fused":
        return rand((B, N, 3, H, D), dtype, seed, 1.5)[:, :, 1].transpose(1, 2)
    if kind == "rows":                      # rows of a longer packed tensor
        return rand((B, H, N + 13, D), dtype, seed, 1.5)[:, :, 5:5 + N]
    return rand((B, 1, N, D), dtype, seed, 1.5).expand(B, H, N, D)      # one head, repeated


QK_CASES = [
    # B, H, N, D, dtype, layout, norm, weight, dims, halves
    (1, 1, 1, 128, "bf16", "heads", True, "shared", (128,), False),
    (1, 3, 1, 64, "fp16", "fused", True, "head", (16, 24, 24), True),
    (2, 5, 33, 128, "bf16", "fused", True, "head", (16, 56, 56), False),
    (2, 2, 67, 128, "bf16", "rows", True, "shared", (16, 56, 56), True),
    (1, 2, 192, 64, "fp32", "heads", False, None, (24, 20, 20), False),
    (3, 4, 17, 64, "fp32", "rows", True, "shared", (16, 16), True),      # half the head turns
    (1, 7, 129, 128, "fp16", "heads", True, None, (8,), False),
    (1, 2, 50, 256, "bf16", "fused", True, "shared", (256,), True),
    (1, 2, 50, 96, "bf16", "heads", True, "head", (32, 32, 32), True),   # lanes left over
    (2, 3, 40, 80, "fp32", "fused", True, "head", (16, 16), False),
    (1, 2, 31, 8, "fp16", "heads", True, "shared", (8,), False),
    (1, 3, 31, 24, "bf16", "heads", True, "shared", None, False),        # norm alone
    (1, 4, 300, 128, "bf16", "repeat", True, "shared", (64,), True),
    (1, 56, 130, 128, "bf16", "fused", True, "shared", (16, 56, 56), False),
]


@pytest.mark.parametrize("case", QK_CASES)
def test_qk_norm_rope(case):
    B, H, N, D, dtype, kind, norm, weight, dims, halves = case
    q, k = layout(kind, B, H, N, D, dtype, 1), layout(kind, B, H, N, D, dtype, 2)
    wq = wk = None
    if weight:
        shape = (H, D) if weight == "head" else (D,)
        wq, wk = rand(shape, dtype, 3, 0.2, 1.0), rand(shape, dtype, 4, 0.2, 1.0)
    table = table_for(N, dims, 5) if dims else None
    qo, ko = T.qk_norm_rope(q, k, wq, wk, eps=1e-5, norm=norm, table=table,
                            pairing="halves" if halves else "interleaved")
    cs = np64(table) if dims else None
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        wn = 1.0 if w is None else (np64(w)[:, None, :] if w.dim() == 2 else np64(w))
        value, bound = ref.norm_rope(np64(x), wn, float(np.float32(1e-5)), norm, cs, halves)
        close(y, value, bound, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("halves", [False, True])
def test_qk_norm_rope_in_place_and_gaps(dtype, halves):
    # in place on a fused projection: V's columns and the rows outside the view stay
    B, H, N, D = 2, 3, 37, 128
    buf = rand((B, N + 4, 3, H, D), dtype, 9)
    before = buf.clone()
    q, k = (buf[:, 2:2 + N, i].transpose(1, 2) for i in range(2))
    table = table_for(N, (16, 56, 56), 6, B)                      # a table per branch
    pairing = "halves" if halves else "interleaved"
    want = T.qk_norm_rope(q, k, table=table, pairing=pairing)
    got = T.qk_norm_rope(q, k, table=table, pairing=pairing, q_out=q, k_out=k)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(buf[:, :, 2], before[:, :, 2])
    assert torch.equal(buf[:, :2], before[:, :2]) and torch.equal(buf[:, 2 + N:], before[:, 2 + N:])
    value, bound = ref.norm_rope(np64(before[:, 2:2 + N, 0].transpose(1, 2)), 1.0,
                                 float(np.float32(1e-6)), True, np64(table)[:, None], halves)
    close(got[0], value, bound, dtype)
    # q alone gives the same
    again = before[:, 2:2 + N, 0].transpose(1, 2)
    assert torch.equal(T.qk_norm_rope(again, table=table, pairing=pairing), want[0])


def test_qk_norm_rope_special_rows():
    # a row of zeros stays zero, an infinity or a NaN stays in its own row
    x = rand((1, 2, 20, 64), "bf16", 3)
    x[0, 0, 3] = 0.0
    x[0, 1, 7, 5] = float("inf")
    x[0, 0, 9, 63] = float("nan")
    table = table_for(20, (64,), 2)
    y = T.qk_norm_rope(x, table=table)
    assert bool((y[0, 0, 3] == 0).all())
    bad = torch.isnan(y).any(-1)[0].cpu()
    rows = {(0, 9), (1, 7)}
    assert {(int(h), int(n)) for h, n in bad.nonzero()} == rows
    # large and small values: the norm neither overflows nor vanishes in fp32
    big = rand((1, 1, 4, 64), "bf16", 4) * 1e15
    small = rand((1, 1, 4, 64), "bf16", 4) * 1e-15
    for v in (big, small):
        value, bound = ref.norm_rope(np64(v), 1.0, 0.0, True, None, False)
        close(T.qk_norm_rope(v, eps=0.0), value, bound, "bf16")


# ---------------------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------------------
def linear_inputs(B, N, K, C, dtype, xH, extras):
    x = rand((B, xH, N, K // xH) if xH else (B, N, K), dtype, 11)
    w = rand((C, K), dtype, 12, K ** -0.5)
    o = {"bias": rand((C,), dtype, 13, 0.3) if "b" in extras else None,
         "gate": rand((B, C), dtype, 14, 0.5, 0.5) if "g" in extras else
         (rand((C,), dtype, 14, 0.5, 0.5) if "G" in extras else None),
         "residual": rand((B, N, C), dtype, 15) if "r" in extras else None}
    return x, w, o


def linear_ref(x, w, o, act):
    """[B][N][C] value and bound."""
    x64 = np64(x)
    if x64.ndim == 4:
        x64 = x64.transpose(0, 2, 1, 3).reshape(x64.shape[0], x64.shape[2], -1)
    vals = []
    for b in range(x64.shape[0]):
        g = o["gate"]
        vals.append(ref.linear(
            x64[b], np64(w), None if o["bias"] is None else np64(o["bias"]), act or "none",
            None if g is None else (np64(g)[b] if g.dim() == 2 else np64(g)),
            None if o["residual"] is None else np64(o["residual"][b])))
    return np.stack([v for v, _ in vals]), np.stack([e for _, e in vals])


LINEAR_CASES = [
    # B, N, K, C, dtype, heads of x (0: token-major), extras, activation, heads of y
    (1, 1, 128, 128, "bf16", 0, "", None, None),
    (1, 1, 8, 8, "fp16", 0, "bgr", "silu", None),
    (2, 1, 520, 1000, "bf16", 0, "bg", None, None),
    (3, 5, 256, 136, "fp16", 0, "bgr", "gelu", None),
    (1, 17, 72, 264, "bf16", 0, "b", "gelu_tanh", None),
    (1, 64, 256, 256, "bf16", 2, "bGr", None, None),
    (2, 65, 192, 384, "fp16", 3, "r", None, 6),
    (1, 130, 1024, 128, "bf16", 8, "br", "silu", 1),
    (1, 200, 448, 640, "bf16", 0, "b", None, 5),
    (2, 257, 256, 512, "bf16", 2, "bgr", None, None),
    (1, 300, 104, 776, "fp16", 0, "bg", "gelu", None),
    (1, 513, 640, 264, "bf16", 0, "", "gelu_tanh", None),
    (1, 512, 192, 7168, "bf16", 0, "bgr", "silu", None),     # 208 columns a tile
    (1, 560, 136, 7176, "fp16", 0, "bgr", None, None),       # 160, and a ragged end
    (2, 520, 128, 4600, "bf16", 2, "br", "gelu", None),
    (1, 1000, 512, 1536, "bf16", 4, "bgr", None, None),
    (2, 700, 328, 520, "fp16", 0, "br", "silu", None),
    (1, 2100, 256, 2304, "bf16", 0, "b", None, 18),
    (1, 9001, 72, 9000, "bf16", 0, "bgr", "gelu_tanh", None),
    (1, 1, 4096, 1024, "bf16", 0, "bgr", "silu", 8),
    (1, 16, 2056, 392, "fp16", 0, "br", None, None),
    (5, 3, 1024, 256, "bf16", 8, "bgr", "gelu", 2),
    (2, 31, 2048, 128, "bf16", 16, "bgr", None, None),
    (1, 255, 1024, 640, "fp16", 0, "r", "gelu_tanh", None),
    (1, 255, 2304, 640, "fp16", 0, "r", "gelu_tanh", None),     # streamed with 256 tokens a tile
    (3, 70, 2048, 264, "bf16", 16, "bgr", "silu", None),
    (1, 129, 4096, 136, "bf16", 0, "b", None, None),
    (1, 7, 64, 24000, "bf16", 0, "bg", None, None),
    (2, 5300, 128, 4608, "fp16", 2, "r", None, 36),
    (1, 1, 1, 1, "fp32", 0, "bgr", "gelu", None),
    (2, 33, 67, 101, "fp32", 0, "bgr", "silu", None),
    (1, 192, 128, 512, "fp32", 2, "b", "gelu_tanh", None),
    (3, 70, 129, 66, "fp32", 3, "r", None, 2),
    (1, 5, 2000, 300, "fp32", 0, "bG", None, None),
    (2, 500, 250, 404, "fp32", 0, "bgr", "gelu", None),
    (1, 1500, 131, 1410, "fp32", 0, "bgr", "silu", None),
    (2, 8, 259, 77, "fp32", 7, "bgr", "gelu_tanh", 7),
    (3, 2, 33, 5, "fp32", 0, "g", None, None),
    (1, 3, 640, 129, "fp32", 10, "r", None, 3),
    (2, 9, 1000, 64, "fp32", 8, "b", None, 2),
]


@pytest.mark.parametrize("case", LINEAR_CASES)
def test_linear(case):
    B, N, K, C, dtype, xH, extras, act, yH = case
    x, w, o = linear_inputs(B, N, K, C, dtype, xH, extras)
    y = T.linear(x, w, act=act, heads=yH, **o)
    assert y.shape == ((B, yH, N, C // yH) if yH else (B, N, C))
    value, bound = linear_ref(x, w, o, act)
    if yH:
        value, bound = (a.reshape(B, N, yH, -1).transpose(0, 2, 1, 3) for a in (value, bound))
    close(y, value, bound, dtype)
    assert T.device_status() == 0
    # the same call gives the same bits
    assert torch.equal(T.linear(x, w, act=act, heads=yH, **o), y)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N", [1, 40, 300, 1030])
def test_linear_views_and_gaps(dtype, N):
    # x: columns of a wider stream; residual and y: rows of longer ones, y over the residual;
    # everything outside y's rows and columns stays
    B, K, C = 2, 256, 384
    wide = rand((B, N, K + 64), dtype, 21)
    x = wide[:, :, 32:32 + K]
    w, bias = rand((C, K), dtype, 22, K ** -0.5), rand((C,), dtype, 23)
    buf = rand((B, N + 9, C + 128), dtype, 24)
    before = buf.clone()
    y = buf[:, 4:4 + N, 64:64 + C]
    o = {"bias": bias, "gate": None, "residual": before[:, 4:4 + N, 64:64 + C]}
    value, bound = linear_ref(x, w, o, None)
    got = T.linear(x, w, bias=bias, residual=y, out=y)
    close(got, value, bound, dtype)
    assert T.device_status() == 0
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[:, 4:4 + N, 64:64 + C] = False
    assert torch.equal(buf[keep], before[keep])


@pytest.mark.parametrize("B,N,heads_in", [(1, 20000, 0), (2, 10300, 32)])
def test_linear_of_a_long_sequence(B, N, heads_in):
    # enough rounds of long products for the 512 x 256 tiles; sampled rows, the ragged end among
    # them (20,000 rows end 32 rows into a tile: its second half does not exist)
    K, C = 4096, 8192
    x, w, o = linear_inputs(B, N, K, C, "bf16", heads_in, "bgr")
    y = T.linear(x, w, act="silu", **o)
    assert T.device_status() == 0
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 511, 512, N // 2, N - 33, N - 32, N - 1], device="cuda")
    xs = x[:, :, rows] if heads_in else x[:, rows]
    sampled = dict(o, residual=o["residual"][:, rows])
    value, bound = linear_ref(xs, w, sampled, "silu")
    close(y[:, rows], value, bound, "bf16")
    assert bool(torch.isfinite(y).all())


def on_gpu(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", [None, "gelu", "gelu_tanh", "silu"])
def test_linear_of_a_long_sequence_in_every_form(dtype, act):
    # the 512 x 256 tiles of every type and activation; sampled rows and columns
    N, K, C = 20000, 4096, 8192
    x, w = on_gpu((1, N, K), dtype, 61), on_gpu((C, K), dtype, 62, K ** -0.5)
    o = {"bias": rand((C,), dtype, 63, 0.3), "gate": rand((1, C), dtype, 64, 0.5, 0.5),
         "residual": on_gpu((1, N, C), dtype, 65)}
    y = T.linear(x, w, act=act, **o)
    assert T.device_status() == 0
    rows = torch.tensor([0, 127, 128, 255, 256, 511, 512, N // 2, N - 33, N - 32, N - 1], device="cuda")
    cols = torch.cat([torch.arange(c, c + 24, device="cuda") for c in (0, 120, 250, 4000, C - 24)])
    part = {"bias": o["bias"][cols], "gate": o["gate"][:, cols],
            "residual": o["residual"][:, rows][:, :, cols]}
    value, bound = linear_ref(x[:, rows], w[cols], part, act)
    close(y[:, rows][:, :, cols], value, bound, dtype)
    assert bool(torch.isfinite(y).all())


@pytest.mark.parametrize("N,C", [(64, 7168), (566, 7168), (20000, 8192)])
def test_sums_lose_nothing_systematically(N, C):
    # 7,168 products through fp16 against 64 bits.  The last rounding is exactly that of the exact
    # value but for its ties, so what goes beyond it comes from the sums: 448 steps of 16 products,
    # each of which may cut off up to two units (2^-23) of a partial sum no larger, on average, than
    # the result.  As a mean over the signs this is 1.1e-4 of the mean magnitude, an order below
    # what the elementwise bound lets pass, and the last rounding averages out (below 1e-6 here).
    K = 7168
    x, w = on_gpu((N, K), "fp16", 71), on_gpu((C, K), "fp16", 72, K ** -0.5)
    y = T.linear(x, w)
    assert T.device_status() == 0
    rows = torch.arange(0, N, max(1, N // 512), device="cuda")
    exact = x[rows].double() @ w.double().t()
    err, rounding = y[rows].double() - exact, exact.half().double() - exact
    lost = K // 16 * 2 * 2.0 ** -23
    assert abs(float((err * exact.sign()).mean() / exact.abs().mean())) <= lost + 2e-6
    rms = lambda t: float(t.square().mean().sqrt())
    assert rms(err) <= rms(rounding) + lost * rms(exact)


def test_linear_keeps_bad_rows_apart():
    # infinities and NaN of one token stay in its row
    for N in (6, 300):
        x, w, _ = linear_inputs(1, N, 256, 512, "bf16", 0, "")
        x[0, 3, 10] = float("nan")
        x[0, 4, 11] = float("inf")
        y = T.linear(x, w)
        ok = torch.isfinite(y).all(-1)[0]
        assert not ok[3] and not ok[4] and int(ok.sum()) == N - 2


TAILS = [-0.25, -1.0, -3.0, -5.0, -7.5, -8.0, -10.5, -12.75, -20.0, -41.0, -42.0, -50.0, -80.0, -100.0,
         -1e4, -1e10, -1e16, -1e20, -1e25, -3e38, 0.0, 0.5, 5.0, 13.0, 60.0, 1e4, 1e20, 3e38]


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
@pytest.mark.parametrize("N", [1, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_activations_keep_their_tails(dtype, N, act):
    # x picks one column of w, so the pre-activations are w's values exactly; every value lies
    # beside an ordinary one, an infinity and a NaN (two columns may be worked on together)
    v = torch.tensor(TAILS).to(DT[dtype]).float()
    v = v[torch.isfinite(v)]
    beside = [v, torch.ones_like(v), v, torch.full_like(v, float("nan")), v, torch.full_like(v, float("inf")),
              v, torch.full_like(v, -float("inf"))]
    cols = torch.stack(beside, 1).reshape(-1)
    w = torch.zeros(len(cols), 64)
    w[:, 7] = cols
    x = torch.zeros(1, N, 64)
    x[:, :, 7] = 1.0
    y = T.linear(x.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), act=act)
    assert T.device_status() == 0
    got = np64(y)[0].reshape(N, len(v), 8)
    value, rel = ref.activation(np64(v), act)
    # fp32 results below its smallest normal number are cut to zero, the output's own steps end too
    step = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}[dtype]
    bound = np.abs(value) * rel + np.abs(np64(v)) * 2.0 ** -125
    tol = bound + torch.finfo(DT[dtype]).eps / 2 * (np.abs(value) + bound) + step / 2
    for i in (0, 2, 4, 6):
        assert np.all(np.abs(got[:, :, i] - value) <= tol), (i, got[0, :, i], value)
    one, rel1 = ref.activation(np.ones(1), act)
    assert np.all(np.abs(got[:, :, 1] - one) <= one * (rel1 + torch.finfo(DT[dtype]).eps))
    assert np.all(np.isnan(got[:, :, 3])) and np.all(np.isposinf(got[:, :, 5]))
    assert not np.any(np.isinf(got[:, :, 7]))            # -infinity times 0, or the limit


# ---------------------------------------------------------------------------------------
# qkv_project
# ---------------------------------------------------------------------------------------
QKV_CASES = [
    # B, N, K, H, D, dtype, heads of x, bias, norm, weight, dims, halves
    (1, 40, 72, 2, 24, "fp32", 0, True, True, "shared", (8, 16), False),
    (2, 9, 128, 3, 64, "fp32", 2, False, True, "head", (16, 24, 24), True),
    (1, 1, 128, 2, 128, "bf16", 0, True, True, "shared", (16, 56, 56), False),
    (2, 1, 72, 3, 64, "fp16", 0, True, True, "head", (64,), True),
    (3, 7, 264, 1, 128, "bf16", 0, False, True, None, (16, 16), True),
    (1, 33, 200, 5, 64, "bf16", 0, True, False, None, (24, 20, 20), False),
    (1, 128, 256, 2, 128, "fp16", 2, True, True, "shared", None, False),
    (1, 100, 256, 2, 128, "fp16", 0, True, False, None, None, False),      # neither: plain products
    (2, 300, 320, 4, 128, "bf16", 5, True, True, "head", (16, 56, 56), True),
    (1, 700, 512, 7, 64, "fp16", 0, True, True, "shared", (16, 16), True),
    (1, 1030, 136, 6, 128, "bf16", 0, True, True, "shared", (44, 42, 42), False),
    (2, 515, 192, 9, 64, "bf16", 0, False, True, "head", (24, 20, 20), False),
    (3, 20, 1024, 3, 64, "bf16", 8, True, True, "head", (48,), True),
    (1, 17, 1032, 4, 128, "fp16", 0, True, True, "shared", (40,), False),
    (2, 120, 512, 2, 128, "bf16", 0, True, False, None, (96,), True),
    (2, 120, 2048, 2, 128, "bf16", 0, True, True, "head", (96,), True),
    (1, 250, 2056, 3, 64, "fp16", 0, True, True, "shared", (64,), False),
    (1, 16, 192, 40, 64, "bf16", 0, False, True, "shared", (16, 24, 24), False),
    (1, 2100, 128, 7, 128, "fp16", 0, True, True, "shared", (16, 56, 56), True),
    (1, 8200, 64, 17, 128, "bf16", 0, True, True, "head", (44, 42, 42), False),
    (2, 4700, 64, 33, 64, "bf16", 0, True, True, "shared", (16, 16), True),
]


def qkv_check(case):
    B, N, K, H, D, dtype, xH, with_bias, norm, weight, dims, halves = case
    x = rand((B, xH, N, K // xH) if xH else (B, N, K), dtype, 31)
    w = rand((3 * H * D, K), dtype, 32, K ** -0.5)
    bias = rand((3 * H * D,), dtype, 33, 0.3) if with_bias else None
    wq = wk = None
    if weight:
        shape = (H, D) if weight == "head" else (D,)
        wq, wk = rand(shape, dtype, 34, 0.2, 1.0), rand(shape, dtype, 35, 0.2, 1.0)
    table = table_for(N, dims, 36) if dims else None
    # outputs: rows of longer packed tensors, as another stream's tokens sit beside these
    packed = [rand((B, H, N + 6, D), dtype, 37 + i) for i in range(3)]
    before = [t.clone() for t in packed]
    out = T.qkv_project(x, w, H, bias, wq, wk, eps=1e-6, norm=norm, table=table,
                        pairing="halves" if halves else "interleaved",
                        out=[t[:, :, 2:2 + N] for t in packed])
    assert T.device_status() == 0
    for t, b in zip(packed, before):
        assert torch.equal(t[:, :, :2], b[:, :, :2]) and torch.equal(t[:, :, 2 + N:], b[:, :, 2 + N:])
    x64 = np64(x)
    if xH:
        x64 = x64.transpose(0, 2, 1, 3).reshape(B, N, K)
    cs = np64(table) if dims else None
    for b in range(B):
        v, e = ref.product(x64[b], np64(w), None if bias is None else np64(bias))
        v, e = (a.reshape(N, 3, H, D).transpose(1, 2, 0, 3) for a in (v, e))
        for i, wt in enumerate((wq, wk, None)):
            if i == 2:
                value, bound = v[i], e[i]
            else:
                wn = 1.0 if wt is None else (np64(wt)[:, None, :] if wt.dim() == 2 else np64(wt))
                value, bound = ref.norm_rope(v[i], wn, float(np.float32(1e-6)), norm, cs, halves,
                                             e[i])
            close(out[i][b], value, bound, dtype)


@pytest.mark.parametrize("halves", [False, True])
def test_qkv_project_of_a_long_sequence(halves):
    # the 512 x 256 tiles; sampled rows
    N, K, H, D = 20100, 4096, 21, 128
    x = rand((1, N, K), "bf16", 51)
    w = rand((3 * H * D, K), "bf16", 52, K ** -0.5)
    bias = rand((3 * H * D,), "bf16", 53, 0.3)
    wq = rand((D,), "bf16", 54, 0.2, 1.0)
    table = table_for(N, (16, 56, 56), 55)
    out = T.qkv_project(x, w, H, bias, wq, wq, table=table,
                        pairing="halves" if halves else "interleaved")
    assert T.device_status() == 0
    rows = torch.tensor([0, 31, 32, 255, 256, 511, 512, N // 2, N - 132, N - 2, N - 1], device="cuda")
    v, e = ref.product(np64(x[0, rows]), np64(w), np64(bias))
    v, e = (a.reshape(len(rows), 3, H, D).transpose(1, 2, 0, 3) for a in (v, e))
    for i in range(3):
        value, bound = (v[i], e[i]) if i == 2 else ref.norm_rope(
            v[i], np64(wq), float(np.float32(1e-6)), True, np64(table[rows]), halves, e[i])
        close(out[i][0][:, rows], value, bound, "bf16")
        assert bool(torch.isfinite(out[i]).all())


def test_qkv_project_of_a_long_sequence_fp16():
    N, K, H, D = 20100, 4096, 21, 128
    x, w = on_gpu((1, N, K), "fp16", 81), on_gpu((3 * H * D, K), "fp16", 82, K ** -0.5)
    wq = rand((H, D), "fp16", 83, 0.2, 1.0)
    table = table_for(N, (16, 24, 24), 84)
    out = T.qkv_project(x, w, H, None, wq, wq, table=table, pairing="halves")
    assert T.device_status() == 0
    rows = torch.tensor([0, 31, 32, 255, 256, 511, 512, N // 2, N - 132, N - 1], device="cuda")
    v, e = ref.product(np64(x[0, rows]), np64(w), None)
    v, e = (a.reshape(len(rows), 3, H, D).transpose(1, 2, 0, 3) for a in (v, e))
    for i in range(3):
        value, bound = (v[i], e[i]) if i == 2 else ref.norm_rope(
            v[i], np64(wq)[:, None, :], float(np.float32(1e-6)), True, np64(table[rows]), True, e[i])
        close(out[i][0][:, rows], value, bound, "fp16")
        assert bool(torch.isfinite(out[i]).all())


@pytest.mark.parametrize("case", QKV_CASES)
def test_qkv_project(case):
    qkv_check(case)


# ---------------------------------------------------------------------------------------
# together, and around them: graphs, streams, offsets past 32 bits, the status word
# ---------------------------------------------------------------------------------------
def shot(N_text, frames, rows, cols, seed):
    """A packed shot of text and video with its metadata, positions and workload."""
    import workloads as W
    tokens = rows * cols
    w = W.custom("layer%d" % seed, B=1, H=3, D=128, dtype="bf16", segments=[
        W.Segment(W.TEXT, 1, N_text), W.Segment(W.PICTURE, 1, 48, pic=1),
        W.Segment(W.TARGET, frames, tokens, frame_dt_s=4 / 24, mask=W.uniform_mask(seed, tokens)),
        W.Segment(W.GUIDE, frames, tokens, frame_dt_s=4 / 24)],
        params=W.Params(gain=(1.25,) + (1.0,) * 8), seed_index=700 + seed)
    video = dict(frame_step=(4 / 24, 0, 0))
    pos = T.pack_token_positions([
        T.TokenGrid(N_text), T.TokenGrid(1, 6, 8, origin=(N_text, 0, 0)),
        T.TokenGrid(frames, rows, cols, origin=(N_text + 1, 0, 0), **video),
        T.TokenGrid(frames, rows, cols, origin=(N_text + 1, 0, 0), **video)])
    assert len(pos) == w.N
    return w, torch.from_numpy(pos).cuda()


class Layer:
    """One joint attention layer: text and the rest of the sequence have their own projections,
    write rows of one packed q, k, v, attend jointly and return through their own output
    projections with a gated residual."""

    def __init__(self, w, pos, seed):
        self.w, H, D = w, w.H, w.D
        self.n_text = w.segments[0].length
        self.C = H * D
        self.x = rand((1, w.N, self.C), "bf16", seed)
        self.part = []
        for i in range(2):
            self.part.append(dict(
                w_qkv=rand((3 * self.C, self.C), "bf16", seed + 10 + i, self.C ** -0.5),
                b_qkv=rand((3 * self.C,), "bf16", seed + 20 + i, 0.2),
                wq=rand((D,), "bf16", seed + 30 + i, 0.1, 1.0),
                wk=rand((D,), "bf16", seed + 40 + i, 0.1, 1.0),
                w_out=rand((self.C, self.C), "bf16", seed + 50 + i, self.C ** -0.5),
                b_out=rand((self.C,), "bf16", seed + 60 + i, 0.2),
                gate=rand((1, self.C), "bf16", seed + 70 + i, 0.3, 0.5)))
        self.meta = T.DeviceMeta(T.pack_token_meta(w.segments), "cuda")
        self.table = T.rope_table(pos, (16, 56, 56))
        self.qkv = [torch.empty((1, H, w.N, D), dtype=torch.bfloat16, device="cuda") for _ in range(3)]
        self.o, self.lse = torch.empty_like(self.qkv[0]), None
        self.lse = torch.empty((1, H, w.N), dtype=torch.float32, device="cuda")
        self.y = torch.empty_like(self.x)

    def rows(self, i):
        return slice(0, self.n_text) if i == 0 else slice(self.n_text, self.w.N)

    def run(self):
        for i, p in enumerate(self.part):
            r = self.rows(i)
            T.qkv_project(self.x[:, r], p["w_qkv"], self.w.H, bias=p["b_qkv"], q_weight=p["wq"],
                          k_weight=p["wk"], table=self.table[r],
                          out=[t[:, :, r] for t in self.qkv])
        T.attn_forward(*self.qkv, self.meta, T.params_from(self.w.params), out=self.o, lse=self.lse)
        for i, p in enumerate(self.part):
            r = self.rows(i)
            T.linear(self.o[:, :, r], p["w_out"], bias=p["b_out"], gate=p["gate"],
                     residual=self.x[:, r], out=self.y[:, r])
        return self.y


@pytest.mark.parametrize("n_text", [40, 300])
def test_a_layer_of_them(n_text):
    from parity_util import compare, run_oracle
    import oracle
    w, pos = shot(n_text, 4, 7, 9, n_text)
    layer = Layer(w, pos, n_text)
    y = layer.run().clone()
    assert T.device_status() == 0
    a = ref.angles(pos.cpu().numpy(), (16, 56, 56), (1e4,) * 3)
    assert np.abs(np64(layer.table) - np.stack([np.cos(a), np.sin(a)], -1)).max() < 4e-7
    H, D = w.H, w.D
    for i, p in enumerate(layer.part):
        r = layer.rows(i)
        x64 = np64(layer.x[0, r])
        v, e = ref.product(x64, np64(p["w_qkv"]), np64(p["b_qkv"]))
        v, e = (t.reshape(len(x64), 3, H, D).transpose(1, 2, 0, 3) for t in (v, e))
        for j, key in enumerate(("wq", "wk", None)):
            value, bound = (v[j], e[j]) if key is None else ref.norm_rope(
                v[j], np64(p[key]), float(np.float32(1e-6)), True, np64(layer.table[r]), False, e[j])
            close(layer.qkv[j][0, :, r], value, bound, "bf16")
        # the output projection of what the attention returned
        o64 = np64(layer.o[0, :, r]).transpose(1, 0, 2).reshape(len(x64), -1)
        value, bound = ref.linear(o64, np64(p["w_out"]), np64(p["b_out"]), "none", np64(p["gate"]),
                                  x64)
        close(y[0, r], value, bound, "bf16")
    rows = oracle.all_rows(1, H, w.N)
    compare(w, layer.o, layer.lse, rows, *run_oracle(w, *layer.qkv, rows), "bf16")


def test_a_captured_layer_replays_on_new_inputs():
    w, pos = shot(40, 3, 6, 8, 3)
    layer = Layer(w, pos, 5)
    want = [layer.run().clone()]                      # also sizes the attention's workspace
    first = layer.x.clone()
    second = rand(tuple(first.shape), "bf16", 99)
    layer.x.copy_(second)
    want.append(layer.run().clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.run()
    for x, y in zip((first, second, first), (want[0], want[1], want[0])):
        layer.x.copy_(x)
        layer.y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, y)


@pytest.mark.parametrize("N", [3, 200, 700])
def test_streams_side_by_side(N):
    # calls on two streams at once, outputs allocated on theirs, give what one stream gives
    x, w, o = linear_inputs(1, N, 512, 768, "bf16", 4, "bgr")
    want = T.linear(x, w, act="silu", **o)
    q = rand((1, 4, N, 128), "bf16", 8)
    table = table_for(N, (64,), 9)
    want_q = T.qk_norm_rope(q, table=table)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            got.append((T.linear(x, w, act="silu", stream=s, **o),
                        T.qk_norm_rope(q, table=table, stream=s)))
    for s in streams:
        s.synchronize()
    for y, z in got:
        assert torch.equal(y, want) and torch.equal(z, want_q)


FIRST_CALL = """
import sys, torch
import video_diffusion_attention_b200 as T
rows = {"few": 3, "many": 300}.get(sys.argv[2], 40)
x = torch.randn(1, rows, 256, device="cuda", dtype=getattr(torch, sys.argv[1]))
w = torch.randn(768, 256, device="cuda").to(x.dtype)
call = {"table": lambda: T.rope_table(torch.ones(40, 2, device="cuda"), (32, 32)),
        "norm": lambda: T.qk_norm_rope(x.view(1, 40, 4, 64).transpose(1, 2)),
        "few": lambda: T.linear(x, w, act="silu"),
        "many": lambda: T.qkv_project(x, w, 4)[0]}[sys.argv[2]]
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    y = call()
graph.replay()
assert torch.equal(y, call()) and T.device_status() == 0
"""


@pytest.mark.parametrize("dtype,what", [("bfloat16", "few"), ("float16", "many"), ("float32", "few"),
                                        ("bfloat16", "norm"), ("float32", "table")])
def test_a_first_call_may_be_captured(dtype, what):
    # a process whose first call of the library is recorded into a graph
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_CALL, dtype, what], cwd=root, check=True, timeout=300)


def test_calls_from_several_threads():
    # the host side keeps what it looks up once a device; every thread has a stream of its own
    import threading
    x, w, o = linear_inputs(1, 300, 512, 768, "fp16", 4, "bgr")
    few = x[:, :, :5]
    few_o = dict(o, residual=o["residual"][:, :5])
    f32 = x.float()
    calls = [lambda: T.linear(x, w, act="silu", **o), lambda: T.linear(few, w, act="gelu", **few_o),
             lambda: T.qkv_project(x, w, 4)[1], lambda: T.qk_norm_rope(x, f32.half())[1],
             lambda: T.qk_norm_rope(f32)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    got, errors = {}, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                got[i] = [[c() for c in calls] for _ in range(20)]
                torch.cuda.current_stream().synchronize()
        except Exception as e:      # raised again below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and len(got) == 4
    for runs in got.values():
        for run in runs:
            assert all(torch.equal(a, b) for a, b in zip(run, want))
    assert T.device_status() == 0


def test_offsets_past_32_bits():
    # more than 2^31 elements: an output of the linear layer, then the norm in place
    N, K, C = 70001, 64, 32768
    x, w, _ = linear_inputs(1, N, K, C, "bf16", 0, "")
    y = T.linear(x, w)
    assert y.numel() > 2 ** 31
    rows = torch.tensor([0, 65535, 65536, 65537, 69887, 70000], device="cuda")
    value, bound = ref.linear(np64(x[0, rows]), np64(w))
    close(y[0, rows], value, bound, "bf16")
    heads = y.view(1, N, 256, 128).transpose(1, 2)
    before = heads[:, :, rows].clone()
    T.qk_norm_rope(heads, q_out=heads)
    value, bound = ref.norm_rope(np64(before), 1.0, float(np.float32(1e-6)), True, None, False)
    close(heads[:, :, rows], value, bound, "bf16")


@pytest.mark.parametrize("N", [4, 300])
def test_launches_skip_while_the_status_word_is_set(N):
    x, w, _ = linear_inputs(1, N, 256, 512, "bf16", 0, "")
    y = torch.full((1, N, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    assert T.device_status() == 0
    T.selftest_wait(5000, arrive=False)
    T.linear(x, w, out=y)
    assert T.device_status() == -10
    assert bool((y == 3.0).all())
    value, bound = ref.linear(np64(x[0]), np64(w))
    close(T.linear(x, w, out=y), value, bound, "bf16")


@pytest.mark.parametrize("N,K,C", [(1, 4096, 1024), (40, 2048, 512), (100, 512, 2048), (3, 64, 384)])
def test_a_status_word_that_changes_meanwhile(N, K, C):
    # the word is set by a kernel on another stream, and read and cleared by the host, while calls
    # of few rows start: every 128 columns of an output are either all there or untouched
    x, w, _ = linear_inputs(1, N, K, C, "bf16", 0, "")
    want = T.linear(x, w)
    assert T.device_status() == 0
    outs = torch.full((6, 40, 1, N, C), 3.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    here, there = torch.cuda.Stream(), torch.cuda.Stream()
    seen = []
    for ys in outs:
        T.selftest_wait(200, arrive=False, stream=there)
        for y in ys:
            T.linear(x, w, out=y, stream=here)
        seen.append(T.device_status(stream=there))       # waits for that stream only
    torch.cuda.synchronize()
    T.device_status()
    assert -10 in seen
    tiles = outs.view(-1, N, C // 128, 128)
    done = (tiles == want.view(N, C // 128, 128)).all(-1).all(1)
    untouched = (tiles == 3.0).all(-1).all(1)
    assert bool((done | untouched).all())
    assert torch.equal(T.linear(x, w), want) and T.device_status() == 0


def test_the_binding_refuses():
    x, w, o = linear_inputs(1, 6, 64, 128, "bf16", 0, "bgr")
    bad = [
        lambda: T.linear(x, w.t()), lambda: T.linear(x, w[:, :32]), lambda: T.linear(x, w.float()),
        lambda: T.linear(x, w, bias=o["bias"][:64]), lambda: T.linear(x, w, act="relu"),
        lambda: T.linear(x, w, bias=o["bias"].float()), lambda: T.linear(x, w, heads=3),
        lambda: T.linear(x.transpose(1, 2), w), lambda: T.linear(x[None, None], w),
        lambda: T.linear(x, w, out=torch.empty(1, 6, 64, dtype=x.dtype, device="cuda")),
        lambda: T.linear(x, w.cpu()), lambda: T.qkv_project(x, w, 3),
        lambda: T.qkv_project(x, w[:96], 1, norm=False, q_weight=o["bias"][:32]),
        lambda: T.qk_norm_rope(x), lambda: T.qk_norm_rope(x[None], table=table_for(5, (64,), 1)),
        lambda: T.qk_norm_rope(x[None], k_out=x[None]),
        lambda: T.qk_norm_rope(x[None], norm=False, q_weight=o["bias"][:64]),
        lambda: T.qk_norm_rope(x[None], pairing="thirds", table=table_for(6, (64,), 1)),
        lambda: T.rope_table(x[0].float(), (64,)), lambda: T.rope_table(x[0], (64,)),
    ]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()
    for f in (lambda: T.qk_norm_rope(x[None], norm=False), lambda: T.linear(x[:, :1].expand(1, 6, 64), w),
              lambda: T.linear(x, w, out=x)):
        with pytest.raises((T.TaraError, ValueError)):
            f()
    torch.cuda.synchronize()
