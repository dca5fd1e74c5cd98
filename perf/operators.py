"""Cases of the operators around the joint attention: rotary tables of several axes, per-head
query/key norms with the rotation, the linear layer with its epilogue, and the Q/K/V projection.

A case names its operator under "op":

  table   pos [N][axes] -> (cos, sin) of every rotated pair
  qk      q, k [B][H][N][D] -> normalised and rotated q, k as the attention takes them
  linear  x, W -> residual + gate * act(x W^T + bias)
  qkv     x, W -> q, k, v [B][H][N][D]: the projection, the norms and the rotation

`run` is the plain form in elementary torch operations, or (own = True) the framework's call.
Sizes are those of the shots in `workloads` (56 heads of 128, 107,126 packed tokens, 8,704 of the
medium one, 566 audio and 512 text tokens, the fp32 tiny shot) and generic ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # the angles of a whole shot, once per shot
        dict(name="table-shot", op="table", N=107126, dims="16,56,56", theta=10000.0, far=0),
        # a short clip at head dim 64, positions far from the origin: latency counts
        dict(name="table-clip", op="table", N=710, dims="24,20,20", theta=256.0, far=50000),
        # every layer of the 56-head shot, out of a fused token-major projection
        dict(name="qk-shot", op="qk", B=1, H=56, N=107126, D=128, dtype="bf16", src="fused",
             norm=True, weight="shared", dims="16,56,56", pairing="interleaved"),
        # two conditioning branches, half-split pairs, weights per head, an odd length
        dict(name="qk-branches", op="qk", B=2, H=8, N=6711, D=64, dtype="fp16", src="heads",
             norm=True, weight="head", dims="16,24,24", pairing="halves"),
        # the exact fp32 path, rotation alone, the smallest shot: latency counts
        dict(name="qk-tiny", op="qk", B=1, H=2, N=192, D=64, dtype="fp32", src="heads",
             norm=False, weight="none", dims="24,20,20", pairing="interleaved"),
        # one vector per conditioning branch through a wide layer (modulation): weights stream
        dict(name="linear-vector", op="linear", B=2, N=1, H=0, K=7168, C=43008, dtype="bf16",
             bias=True, act="none", gate=False, residual=False),
        # output projection of the text tokens, head-major input, gated residual
        dict(name="linear-text", op="linear", B=1, N=512, H=56, K=7168, C=7168, dtype="bf16",
             bias=True, act="none", gate=True, residual=True),
        # feed-forward of the medium shot
        dict(name="linear-medium", op="linear", B=1, N=8704, H=0, K=1024, C=4096, dtype="fp16",
             bias=True, act="gelu_tanh", gate=False, residual=False),
        # output projection of the 56-head shot
        dict(name="linear-shot", op="linear", B=1, N=107126, H=56, K=7168, C=7168, dtype="bf16",
             bias=True, act="none", gate=True, residual=True),
        # fp32 layer of the smallest shot: latency counts
        dict(name="linear-tiny", op="linear", B=1, N=192, H=0, K=128, C=512, dtype="fp32",
             bias=True, act="silu", gate=False, residual=False),
        # Q, K, V of the audio tokens
        dict(name="qkv-audio", op="qkv", B=1, N=566, H=56, D=128, K=7168, dtype="bf16",
             bias=True, norm=True, dims="16,56,56", pairing="halves"),
        # Q, K, V of the whole shot
        dict(name="qkv-shot", op="qkv", B=1, N=107126, H=56, D=128, K=7168, dtype="bf16",
             bias=True, norm=True, dims="16,56,56", pairing="interleaved"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dims(rng, D):
    """Axis sizes (even, summing to a multiple of 16 at most D)."""
    total = rng.choice([D, D, D, D // 2]) // 2
    cuts = sorted(rng.sample(range(1, total), rng.choice([0, 1, 2, 2, 2])))
    edges = [0] + cuts + [total]
    return ",".join(str(2 * (b - a)) for a, b in zip(edges, edges[1:]))


def draw(rng):
    op = rng.choice(["table", "qk", "qk", "linear", "linear", "linear", "qkv", "qkv"])
    D = rng.choice([64, 128])
    if op == "table":
        return dict(op=op, N=_log(rng, 1, 107126), dims=_dims(rng, D),
                    theta=rng.choice([256.0, 10000.0, 1000000.0]), far=rng.choice([0, 0, 50000]))
    B = rng.choice([1, 1, 2, 3])
    pairing = rng.choice(["interleaved", "halves"])
    if op == "qk":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        H = _log(rng, 1, 56)
        N = _log(rng, 1, 107126 * 28 // (B * H) if B * H > 28 else 107126)
        norm = rng.random() < 0.8
        return dict(op=op, B=B, H=H, N=N, D=D, dtype=dtype, src=rng.choice(["fused", "heads"]),
                    norm=norm, weight=rng.choice(["shared", "head"]) if norm else "none",
                    dims=_dims(rng, D), pairing=pairing)
    if op == "qkv":
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        H = _log(rng, 2, 56)
        return dict(op=op, B=B, N=_log(rng, 1, 20000) // B + 1, H=H, D=D, K=8 * _log(rng, 8, 896),
                    dtype=dtype, bias=rng.random() < 0.7, norm=rng.random() < 0.8,
                    dims=_dims(rng, D), pairing=pairing)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    big = dtype != "fp32"
    H = rng.choice([0, _log(rng, 1, 56 if big else 8)])
    K = H * D if H else 8 * _log(rng, 8, 1792 if big else 128)
    return dict(op=op, B=B, N=_log(rng, 1, 30000 if big else 4000) // B + 1, H=H, K=K,
                C=8 * _log(rng, 8, 2688 if big else 256), dtype=dtype, bias=rng.random() < 0.7,
                act=rng.choice(["none", "gelu", "gelu_tanh", "silu"]), gate=rng.random() < 0.4,
                residual=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _axes(case):
    return [int(d) for d in case["dims"].split(",")]


def _positions(N, axes, far, g):
    """Positions of a packed shot on the GPU: a run of text on the first axis, then frames of a
    40 x 50 patch grid whose clock starts behind the text; `far` moves the clock away from 0."""
    i = torch.arange(N, device="cuda", dtype=torch.float64)
    text = min(512, N // 4)
    f = torch.clamp(i - text, min=0)
    start = torch.rand((), generator=g, device="cuda", dtype=torch.float64)
    t = torch.where(i < text, i, text + torch.floor(f / 2000) * (4.0 / 24.0)) + start + far
    h = torch.where(i < text, torch.zeros_like(i), torch.floor(f / 50) % 40)
    w = torch.where(i < text, torch.zeros_like(i), f % 50)
    return torch.stack([t, h, w][:axes], dim=1).to(torch.float32).contiguous()


def _randn(shape, dtype, g, scale=1.0, shift=0.0):
    x = torch.empty(shape, dtype=dtype, device="cuda")
    flat = x.view(-1)
    step = 1 << 28
    for a in range(0, flat.numel(), step):      # in pieces: no fp32 copy of a whole tensor
        n = min(step, flat.numel() - a)
        piece = torch.randn(n, generator=g, device="cuda", dtype=torch.float32)
        flat[a:a + n].copy_(piece.mul_(scale).add_(shift))
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    axes = _axes(case) if "dims" in case else None
    if op == "table":
        s["pos"] = _positions(case["N"], len(axes), case["far"], g)
        if own:
            import video_diffusion_attention_b200 as T
            s["T"] = T
        return s
    dt = DTYPES[case["dtype"]]
    B, N = case["B"], case["N"]
    if op in ("qk", "qkv"):
        H, D = case["H"], case["D"]
        # the table a program computes once per shot
        a = _angles(_positions(N, len(axes), 0, g), axes, 10000.0)
        s["table"] = torch.stack([torch.cos(a), torch.sin(a)], dim=-1).to(torch.float32)
        wshape = (H, D) if case.get("weight") == "head" else (D,)
        s["wq"] = s["wk"] = None
        if case["norm"]:
            s["wq"] = _randn(wshape, dt, g, 0.1, 1.0)
            s["wk"] = _randn(wshape, dt, g, 0.1, 1.0)
    if op == "qk":
        if case["src"] == "fused":      # token-major output of one projection
            buf = _randn((B, N, 3, H, D), dt, g, 1.5)
            s["q"], s["k"] = buf[:, :, 0].transpose(1, 2), buf[:, :, 1].transpose(1, 2)
        else:
            s["q"], s["k"] = _randn((B, H, N, D), dt, g, 1.5), _randn((B, H, N, D), dt, g, 1.5)
    elif op == "qkv":
        C = 3 * H * D
        s["x"] = _randn((B, N, case["K"]), dt, g)
        s["w"] = _randn((C, case["K"]), dt, g, case["K"] ** -0.5)
        s["bias"] = _randn((C,), dt, g, 0.2) if case["bias"] else None
    else:
        H, K, C = case["H"], case["K"], case["C"]
        s["x"] = _randn((B, H, N, K // H) if H else (B, N, K), dt, g)
        s["w"] = _randn((C, K), dt, g, K ** -0.5)
        s["bias"] = _randn((C,), dt, g, 0.2) if case["bias"] else None
        s["gate"] = _randn((B, C), dt, g, 0.3, 0.5) if case["gate"] else None
        s["residual"] = _randn((B, N, C), dt, g) if case["residual"] else None
    if own:
        import video_diffusion_attention_b200 as T
        s["T"] = T
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _angles(pos, axes, theta):
    """[N][R/2] angles in 64 bits: far positions times frequencies lose their phase in 32."""
    cols = []
    for a, d in enumerate(axes):
        i = torch.arange(d // 2, device=pos.device, dtype=torch.float64)
        cols.append(pos[:, a:a + 1].double() * torch.exp(i * (-2.0 / d * math.log(theta))))
    return torch.cat(cols, dim=1)


def _head_norm(x, w, eps):
    return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + eps) * w


def _rotate(x, table, pairing):
    """x [B][H][N][D], table [N][R/2][2]; the first R columns are rotated."""
    c, s = table[..., 0], table[..., 1]
    R = 2 * c.shape[-1]
    head = x[..., :R]
    if pairing == "interleaved":
        a, b = head[..., 0::2], head[..., 1::2]
        r = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = head[..., :R // 2], head[..., R // 2:]
        r = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return r if R == x.shape[-1] else torch.cat([r, x[..., R:]], dim=-1)


def _norm_rotate(x, w, table, pairing):
    if w is not None:
        x = _head_norm(x, w.float() if w.dim() == 1 else w.float()[:, None, :], 1e-6)
    return _rotate(x, table, pairing)


def _act(x, act):
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.7071067811865476))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(0.7978845608028654 * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "table":
        a = _angles(s["pos"], _axes(case), case["theta"])
        return torch.stack([torch.cos(a), torch.sin(a)], dim=-1).to(torch.float32)
    dt = DTYPES[case["dtype"]]
    if op == "qk":
        return tuple(_norm_rotate(x.float(), w, s["table"], case["pairing"]).to(dt)
                     for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    if op == "qkv":
        B, N, H, D = case["B"], case["N"], case["H"], case["D"]
        y = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        q, k, v = y.view(B, N, 3, H, D).permute(2, 0, 3, 1, 4)
        q = _norm_rotate(q, s["wq"], s["table"], case["pairing"]).to(dt)
        k = _norm_rotate(k, s["wk"], s["table"], case["pairing"]).to(dt)
        return q, k, v.to(dt).contiguous()
    x = s["x"].float()
    if x.dim() == 4:
        x = x.transpose(1, 2).flatten(2)
    y = x @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, case["act"])
    if s["gate"] is not None:
        y = y * s["gate"].float()[:, None, :]
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt)


def _own(s):
    case, T = s["case"], s["T"]
    op = case["op"]
    if op == "table":
        return T.rope_table(s["pos"], _axes(case), case["theta"])
    if op == "qk":
        return T.qk_norm_rope(s["q"], s["k"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6,
                              norm=case["norm"], table=s["table"], pairing=case["pairing"])
    if op == "qkv":
        return T.qkv_project(s["x"], s["w"], case["H"], bias=s["bias"], q_weight=s["wq"],
                             k_weight=s["wk"], eps=1e-6, norm=case["norm"], table=s["table"],
                             pairing=case["pairing"])
    return T.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], gate=s["gate"],
                    residual=s["residual"])


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op = case["op"]
    if op == "table":
        R, A = sum(_axes(case)), len(_axes(case))
        return {"bytes": 4 * case["N"] * (A + R), "flops": 10 * case["N"] * R}
    e = SIZE[case["dtype"]]
    B, N = case["B"], case["N"]
    R = sum(_axes(case)) if "dims" in case else 0
    if op == "qk":
        el = 2 * B * case["H"] * N * case["D"]
        return {"bytes": 2 * el * e + 4 * R * N, "flops": el * (4 * case["norm"] + 3)}
    K = case["K"]
    C = 3 * case["H"] * case["D"] if op == "qkv" else case["C"]
    b = e * (B * N * (K + C) + C * K) + (e * C if case["bias"] else 0)
    if op == "qkv":
        b += 4 * R * N
    else:
        b += e * (B * N * C if case["residual"] else 0) + e * (B * C if case["gate"] else 0)
    return {"bytes": b, "flops": 2 * B * N * K * C}


# ---------------------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_rotary(x, w, angle, halves, out):
    """One head plane [N][D] (fp64) through the norm and the rotation, into out."""
    if w is not None:
        x = x / torch.sqrt(torch.sum(x ** 2, dim=1, keepdim=True) / x.shape[1] + 1e-6) * w
    out.copy_(x)
    P = angle.shape[1]
    j = torch.arange(P, device=x.device)
    ia, ib = (j, j + P) if halves else (2 * j, 2 * j + 1)
    z = torch.complex(x[:, ia], x[:, ib]) * angle
    out[:, ia] = z.real
    out[:, ib] = z.imag


def _exact_heads(x, w, table, halves):
    """x [B][H][N][D] of any type -> fp64, plane by plane."""
    B, H, N, D = x.shape
    t = torch.complex(table[..., 0].double(), table[..., 1].double())
    out = torch.empty((B, H, N, D), dtype=torch.float64, device=x.device)
    for b in range(B):
        for h in range(H):
            wh = None if w is None else (w if w.dim() == 1 else w[h]).double()
            _exact_rotary(x[b, h].double(), wh, t, halves, out[b, h])
    return out


def _exact_rows(x, w, bias):
    """x [M][K] times w [C][K] transposed plus bias, in fp64, in blocks of rows."""
    wd = w.double()
    out = torch.empty((x.shape[0], w.shape[0]), dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[0], 8192):
        torch.matmul(x[a:a + 8192].double(), wd.t(), out=out[a:a + 8192])
    if bias is not None:
        out += bias.double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "table":
        pos = s["pos"].double()
        cols = []
        for a, d in enumerate(_axes(case)):
            f = case["theta"] ** (-torch.arange(0, d, 2, device=pos.device, dtype=torch.float64) / d)
            cols.append(torch.outer(pos[:, a], f))
        z = torch.polar(torch.ones((), dtype=torch.float64, device=pos.device),
                        torch.cat(cols, dim=1))
        return torch.view_as_real(z)
    halves = case.get("pairing") == "halves"
    if op == "qk":
        return tuple(_exact_heads(s[n], s["w" + n], s["table"], halves) for n in "qk")
    if op == "qkv":
        B, N, H, D, K = (case[c] for c in ("B", "N", "H", "D", "K"))
        outs = []
        for part, n in enumerate("qkv"):
            rows = slice(part * H * D, (part + 1) * H * D)
            y = _exact_rows(s["x"].reshape(B * N, K), s["w"][rows],
                            None if s["bias"] is None else s["bias"][rows])
            y = y.view(B, N, H, D).transpose(1, 2)
            outs.append(y.contiguous() if n == "v"
                        else _exact_heads(y, s["w" + n], s["table"], halves))
        return tuple(outs)
    B, N, K, C = case["B"], case["N"], case["K"], case["C"]
    x = s["x"]
    if case["H"]:
        x = x.permute(0, 2, 1, 3)
    y = _exact_rows(x.reshape(B * N, K), s["w"], s["bias"]).view(B, N, C)
    act = case["act"]
    if act == "gelu":           # x Phi(x)
        y = y * (torch.special.erfc(-y / math.sqrt(2.0)) / 2.0)
    elif act == "gelu_tanh":    # the tanh form as a logistic
        y = y * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3))
    elif act == "silu":
        y = y * torch.sigmoid(y)
    if s["gate"] is not None:
        y = y * s["gate"].double().unsqueeze(1)
    if s["residual"] is not None:
        y = y + s["residual"].double()
    return y
