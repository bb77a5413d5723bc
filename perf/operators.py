"""Measured cases of the 8-bit operators: the RMS norm with the residual's
addition, the gated activation, and the FP8 (e4m3) product with a scale per
block of 128, dense and grouped by expert.

The codes of 128 consecutive values v are c = e4m3(v / s) with the float32
scale s = max(max|v| / 448, 2^-126); a weight has one scale per 128 x 128
block.  `run` computes each operator in elementary torch operations in
float32, or calls the library where `own` is true.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step's norm before a 4096-wide attention projection
        {"name": "norm_m1_d4096_fp8", "op": "norm", "M": 1, "D": 4096, "x": "bf16", "w": "bf16",
         "residual": True, "out": "fp8"},
        # a float32 residual stream of a ragged batch before the rotated linear (5120 = 8*8*8*5*2)
        {"name": "norm_m333_d5120_f32_bf16", "op": "norm", "M": 333, "D": 5120, "x": "f32",
         "w": "f32", "residual": True, "out": "bf16"},
        # prefill of 8192 tokens, 8192 wide
        {"name": "norm_m8192_d8192_fp8", "op": "norm", "M": 8192, "D": 8192, "x": "bf16",
         "w": "bf16", "residual": True, "out": "fp8"},
        # decode batch between the MLP's products, 11008 = 86 blocks
        {"name": "silu_m16_d11008", "op": "silu", "M": 16, "D": 11008, "x": "bf16"},
        # prefill of 2000 tokens between the products of a 28672-wide MLP
        {"name": "silu_m2000_d28672", "op": "silu", "M": 2000, "D": 28672, "x": "bf16"},
        # decode of one token, attention projection: one pass over 16 MiB of weights
        {"name": "gemm_m1_4096_4096", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "out": "bf16"},
        # decode batch on the widest MLP projection: one pass over 224 MiB of weights
        {"name": "gemm_m16_8192_28672", "op": "gemm", "M": 16, "N": 28672, "K": 8192,
         "out": "bf16"},
        # a ragged chunk of prefill, float32 output for the next step's sum
        {"name": "gemm_m200_4096_11008_f32", "op": "gemm", "M": 200, "N": 11008, "K": 4096,
         "out": "f32"},
        # prefill of 4096 tokens: matrix-core bound
        {"name": "gemm_m4096_8192_28672", "op": "gemm", "M": 4096, "N": 28672, "K": 8192,
         "out": "bf16"},
        # decode of 8 tokens, 8 of 64 experts each: gate and up, rows read by index
        {"name": "grouped_e64_m64_4096_4096", "op": "grouped", "E": 64, "tokens": 8, "top": 8,
         "N": 4096, "K": 4096, "gather": True, "out": "bf16"},
        # a short ragged batch over few experts, sorted rows, some experts without any
        {"name": "grouped_e16_m500_2048_4096_f32", "op": "grouped", "E": 16, "tokens": 500,
         "top": 1, "N": 4096, "K": 2048, "gather": False, "out": "f32"},
        # prefill of 2048 tokens, 4 of 32 experts each
        {"name": "grouped_e32_m8192_4096_8192", "op": "grouped", "E": 32, "tokens": 2048,
         "top": 4, "N": 8192, "K": 4096, "gather": True, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "silu", "gemm", "gemm", "grouped", "grouped"))
    if op == "norm":
        return {"op": op, "M": _log(rng, 1, 8192), "D": 16 * _log(rng, 16, 512),
                "x": rng.choice(("bf16", "f32")), "w": rng.choice(("bf16", "f32")),
                "residual": rng.random() < 0.8, "out": rng.choice(("fp8", "fp8", "bf16", "f32"))}
    if op == "silu":
        return {"op": op, "M": _log(rng, 1, 2000), "D": 16 * _log(rng, 16, 1792),
                "x": rng.choice(("bf16", "f32"))}
    out = rng.choice(("bf16", "bf16", "f32"))
    if op == "gemm":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 256, 28672),
                "K": 16 * _log(rng, 16, 512), "out": out}
    return {"op": op, "E": _log(rng, 4, 64), "tokens": _log(rng, 1, 2048),
            "top": rng.choice((1, 2, 4)), "N": _log(rng, 512, 4096), "K": 16 * _log(rng, 32, 256),
            "gather": rng.random() < 0.6, "out": out}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _code_rows(v):
    """Codes and scales of the rows of a float32 matrix, a scale per 1 x 128."""
    M, D = v.shape
    B = _blocks(D)
    p = torch.nn.functional.pad(v, (0, B * BLOCK - D)).view(M, B, BLOCK)
    s = (p.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    q = (p / s.unsqueeze(2)).view(M, B * BLOCK)[:, :D].to(torch.float8_e4m3fn)
    return q.contiguous(), s


def _code_weight(w):
    """Codes and scales of a weight [N][K], a scale per 128 x 128."""
    N, K = w.shape
    A, B = _blocks(N), _blocks(K)
    p = torch.nn.functional.pad(w, (0, B * BLOCK - K, 0, A * BLOCK - N))
    s = p.view(A, BLOCK, B, BLOCK).abs().amax((1, 3)) / E4M3_MAX
    q = p.view(A, BLOCK, B, BLOCK) / s.view(A, 1, B, 1)
    return q.view(A * BLOCK, B * BLOCK)[:N, :K].to(torch.float8_e4m3fn), s


def _activations(g, M, D):
    """N(0, 1) with 1 % of the channels 20 times larger."""
    x = torch.randn((M, D), generator=g, device="cuda")
    hot = torch.rand((D,), generator=g, device="cuda") < 0.01
    return x * torch.where(hot, 20.0, 1.0)


def _route(case, seed):
    """A router's choice: every token takes its `top` best experts, and some experts are liked
    more.  The expert of every (token, choice), and the rows of each expert."""
    g = torch.Generator().manual_seed(int(seed))
    E = case["E"]
    score = torch.randn((E,), generator=g) + torch.randn((case["tokens"], E), generator=g)
    expert = score.topk(min(case["top"], E), dim=1).indices.flatten()
    return expert, torch.bincount(expert, minlength=E)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": case}
    op = case["op"]
    if op == "norm":
        M, D, dt = case["M"], case["D"], DTYPES[case["x"]]
        st["x"] = torch.randn((M, D), generator=g, device="cuda").to(dt)
        if case["residual"]:
            st["residual"] = (4 * _activations(g, M, D)).to(dt)
            st["residual_out"] = torch.empty((M, D), dtype=dt, device="cuda")
        st["w"] = (1 + 0.2 * torch.randn((D,), generator=g, device="cuda")).to(DTYPES[case["w"]])
        if case["out"] == "fp8":
            st["q"] = torch.empty((M, D), dtype=torch.float8_e4m3fn, device="cuda")
            st["s"] = torch.empty((M, _blocks(D)), device="cuda")
        else:
            st["y"] = torch.empty((M, D), dtype=DTYPES[case["out"]], device="cuda")
        return st
    if op == "silu":
        M, D = case["M"], case["D"]
        st["x"] = (2 * torch.randn((M, 2 * D), generator=g, device="cuda")).to(DTYPES[case["x"]])
        st["q"] = torch.empty((M, D), dtype=torch.float8_e4m3fn, device="cuda")
        st["s"] = torch.empty((M, _blocks(D)), device="cuda")
        return st
    N, K = case["N"], case["K"]
    E = case.get("E", 1)
    st["w"] = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device="cuda")
    st["ws"] = torch.empty((E, _blocks(N), _blocks(K)), device="cuda")
    for e in range(E):
        st["w"][e], st["ws"][e] = _code_weight(
            0.02 * torch.randn((N, K), generator=g, device="cuda"))
    if op == "gemm":
        M = rows = case["M"]
    else:
        expert, count = _route(case, seed)
        order = torch.argsort(expert, stable=True).cuda()
        M = expert.numel()
        st["offsets"] = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
        st["offsets"][1:] = count.cumsum(0)
        st["sizes"] = count.tolist()
        rows = M
        if case["gather"]:
            rows = case["tokens"]
            st["rows"] = (order // (M // rows)).to(torch.int32)
    st["a"], st["as"] = _code_rows(_activations(g, rows, K))
    st["y"] = torch.empty((M, N), dtype=DTYPES[case["out"]], device="cuda")
    if own:
        import rotated_bit_amd as H
        st["W"] = H.FP8Weight(st["w"], st["ws"])
    return st


def _values(q, s, rows_per_scale):
    """The float32 values of codes [R][K] with a scale per rows_per_scale x 128."""
    R, K = q.shape
    s = s.repeat_interleave(rows_per_scale, 0)[:R] if rows_per_scale > 1 else s
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :K]


def run(state):
    case = state["case"]
    if own:
        return _run_own(case["op"], state)
    op = case["op"]
    if op == "norm":
        h = state["x"].float()
        if case["residual"]:
            h = h + state["residual"].float()
        y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * state["w"].float()
        got = {"residual": h.to(state["x"].dtype)} if case["residual"] else {}
        if case["out"] == "fp8":
            got["codes"], got["scales"] = _code_rows(y)
        else:
            got["y"] = y.to(DTYPES[case["out"]])
        return got
    if op == "silu":
        D = case["D"]
        gate, up = state["x"][:, :D].float(), state["x"][:, D:].float()
        q, s = _code_rows(gate / (1 + torch.exp(-gate)) * up)
        return {"codes": q, "scales": s}
    a = _values(state["a"], state["as"], 1)
    if op == "gemm":
        return (a @ _values(state["w"][0], state["ws"][0], BLOCK).T).to(DTYPES[case["out"]])
    if case["gather"]:
        a = a[state["rows"]]
    parts = a.split(state["sizes"])
    return torch.cat([(p @ _values(state["w"][e], state["ws"][e], BLOCK).T)
                      for e, p in enumerate(parts) if p.shape[0]]).to(DTYPES[case["out"]])


def _run_own(op, st):
    import rotated_bit_amd as H
    if op == "norm":
        if "q" in st:
            H.harp_rmsnorm_fp8(st["x"], st["w"], st["q"], st["s"], eps=EPS,
                               residual=st.get("residual"), residual_out=st.get("residual_out"))
            got = {"codes": st["q"], "scales": st["s"]}
        else:
            H.harp_rmsnorm(st["x"], st["w"], st["y"], eps=EPS, residual=st.get("residual"),
                           residual_out=st.get("residual_out"))
            got = {"y": st["y"]}
        if "residual" in st:
            got["residual"] = st["residual_out"]
        return got
    if op == "silu":
        H.harp_silu_mul_fp8(st["x"], st["q"], st["s"])
        return {"codes": st["q"], "scales": st["s"]}
    if op == "gemm":
        H.harp_fp8_gemm(st["W"], st["a"], st["as"], st["y"])
    else:
        H.harp_fp8_gemm_grouped(st["W"], st["a"], st["as"], st["offsets"], st["y"],
                                rows=st.get("rows"))
    return st["y"]


def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    if op == "norm":
        M, D, x = case["M"], case["D"], size[case["x"]]
        out = D + 4 * _blocks(D) if case["out"] == "fp8" else D * size[case["out"]]
        return {"bytes": M * (D * x * (3 if case["residual"] else 1) + out) + D * size[case["w"]],
                "flops": 5 * M * D}
    if op == "silu":
        M, D = case["M"], case["D"]
        return {"bytes": M * (2 * D * size[case["x"]] + D + 4 * _blocks(D)), "flops": 5 * M * D}
    N, K = case["N"], case["K"]
    weight = N * K + 4 * _blocks(N) * _blocks(K)
    row_in, row_out = K + 4 * _blocks(K), N * size[case["out"]]
    if op == "gemm":
        M = case["M"]
        return {"bytes": weight + M * (row_in + row_out), "flops": 2 * M * N * K}
    top = min(case["top"], case["E"])
    M = case["tokens"] * top
    rows = case["tokens"] if case["gather"] else M
    # experts that get a row, on average: the others' weights need not be read
    live = sum(int((_route(case, seed)[1] > 0).sum()) for seed in range(16)) / 16
    return {"bytes": int(live * weight) + rows * row_in + M * row_out + 4 * (M + case["E"] + 1),
            "flops": 2 * M * N * K}


def _exact_codes(v):
    """Scales, and the values that the codes round (float64)."""
    M, D = v.shape
    B = _blocks(D)
    wide = torch.zeros((M, B * BLOCK), dtype=torch.float64, device=v.device)
    wide[:, :D] = v
    wide = wide.reshape(M, B, BLOCK)
    s = torch.maximum(wide.abs().max(dim=2).values / E4M3_MAX,
                      torch.tensor(TINY, dtype=torch.float64, device=v.device))
    return {"codes": (wide / s[:, :, None]).reshape(M, -1)[:, :D], "scales": s}


def _exact_product(a, sa, w, sw):
    """Rows a [R][K] with scales sa [R][B] times w [N][K] with scales sw [N/128][B]."""
    K, N = a.shape[1], w.shape[0]
    k = torch.arange(K, device=a.device) // BLOCK
    n = torch.arange(N, device=a.device) // BLOCK
    a64 = a.to(torch.float64) * sa.to(torch.float64)[:, k]
    w64 = w.to(torch.float64) * sw.to(torch.float64)[n][:, k]
    return torch.mm(a64, w64.t().contiguous())


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].to(torch.float64)
        if case["residual"]:
            h = h + st["residual"].to(torch.float64)
        root = torch.sqrt((h * h).sum(dim=1) / h.shape[1] + EPS)
        y = h / root[:, None] * st["w"].to(torch.float64)
        got = _exact_codes(y) if case["out"] == "fp8" else {"y": y}
        if case["residual"]:
            got["residual"] = h
        return got
    if op == "silu":
        gate, up = st["x"].to(torch.float64).chunk(2, dim=1)
        return _exact_codes(gate * torch.sigmoid(gate) * up)
    if op == "gemm":
        return _exact_product(st["a"], st["as"], st["w"][0], st["ws"][0])
    y = torch.empty(st["y"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for e, size in enumerate(st["sizes"]):
        if size:
            i = torch.arange(at, at + size, device="cuda")
            i = st["rows"][i].long() if case["gather"] else i
            y[at:at + size] = _exact_product(st["a"][i], st["as"][i], st["w"][e], st["ws"][e])
        at += size
    return y
