"""One block of an FP8 checkpoint around its matrix products, as cases to measure.

Four operators, in the order in which a block uses them:
 - norm: residual add of a block's output (with its own norm, gate and scale), then the next block's norm, written as
   bf16 or as 8-bit activations with a scale for each token and 128 channels;
 - encode: the same 8-bit activations from rows that no norm precedes (attention's output);
 - gemm: 8-bit activations times 8-bit weights with a scale for each 128 x 128 tile;
 - ffn: the gate and up projections with SiLU(gate) * up, one call, h in bf16 or as the down projection's 8-bit input.

Each has a plain form in elementary torch operations (32-bit arithmetic, rounded once), the framework's call (`own`),
and `exact`, the definition in 64 bits written apart from the plain form.
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # smallest scale: the smallest normal fp32


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token: fp32 rows as a projection leaves them, bf16 residual stream, 8-bit output
        dict(name="norm_decode_1", op="norm", T=1, H=4096, x="f32", res="bf16", post=False, gate="none", y="e4m3"),
        # 130 drafted tokens of a small hidden size; a norm after the block, a gate row for all tokens, bf16 output
        dict(name="norm_verify_130", op="norm", T=130, H=2048, x="f32", res="f32", post=True, gate="row", y="bf16"),
        # a prompt of 8191 tokens, everything bf16, a gate for each token, 8-bit output
        dict(name="norm_prompt_8191", op="norm", T=8191, H=4096, x="bf16", res="bf16", post=True, gate="full",
             y="e4m3"),
        # attention's output of 16 drafted tokens, ahead of the output projection
        dict(name="encode_verify_16", op="encode", T=16, K=4096, x="bf16"),
        # the down projection's input of a prompt, fp32 rows
        dict(name="encode_prompt_4099", op="encode", T=4099, K=12288, x="f32"),
        # one decoded token through a fused projection: the weights' one read
        dict(name="gemm_decode_1", op="gemm", T=1, M=12288, K=4096, y="f32"),
        # 17 drafted tokens through a down projection
        dict(name="gemm_verify_17", op="gemm", T=17, M=4096, K=12288, y="f32"),
        # a chunk of 333 tokens, a ragged number of rows
        dict(name="gemm_chunk_333", op="gemm", T=333, M=4870, K=4096, y="bf16"),
        # a prompt of 8192 tokens
        dict(name="gemm_prompt_8192", op="gemm", T=8192, M=12288, K=4096, y="bf16"),
        # a shared expert of a decode batch
        dict(name="ffn_decode_8", op="ffn", T=8, I=512, K=2048, h="bf16"),
        # 64 drafted tokens through a dense feed-forward block, h for the down projection
        dict(name="ffn_verify_64", op="ffn", T=64, I=12288, K=4096, h="e4m3"),
        # a prompt of 4099 tokens
        dict(name="ffn_prompt_4099", op="ffn", T=4099, I=12288, K=4096, h="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    """One more case of the listed ranges: one token to thousands, small and large matrices, ragged sizes."""
    op = rng.choice(["norm", "encode", "gemm", "ffn"])
    if op == "norm":
        H = 16 * _log_int(rng, 4, 768)
        return dict(op=op, T=_log_int(rng, 1, min(16384, 8191 * 4096 // H)), H=H, x=rng.choice(["f32", "bf16"]),
                    res=rng.choice(["f32", "bf16"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "row", "full"]), y=rng.choice(["bf16", "e4m3"]))
    K = 16 * _log_int(rng, 8, 768)
    if op == "encode":
        return dict(op=op, T=_log_int(rng, 1, min(16384, 4099 * 12288 // K)), K=K, x=rng.choice(["f32", "bf16"]))
    if op == "gemm":
        M = _log_int(rng, 64, 16384)
        return dict(op=op, T=_log_int(rng, 1, min(8192, 8192 * 12288 * 4096 // (M * K))), M=M, K=K,
                    y=rng.choice(["f32", "bf16"]))
    I = _log_int(rng, 64, 12288)
    return dict(op=op, T=_log_int(rng, 1, min(8192, 4099 * 12288 * 4096 // (I * K))), I=I, K=K,
                h=rng.choice(["f32", "bf16", "e4m3"]))


# ---------------------------------------------------------------- inputs
_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _weight(M, K, g):
    """E4M3 weights [M][K] of a random matrix, one fp32 scale for each 128 x 128 tile, as a checkpoint holds them."""
    w = torch.randn(M, K, generator=g, device=DEV)
    w *= (0.5 + torch.rand(M, 1, generator=g, device=DEV)) / math.sqrt(K)
    Mb, Kb = -(-M // 128), -(-K // 128)
    full = torch.zeros(Mb * 128, Kb * 128, device=DEV)
    full[:M, :K] = w
    tiles = full.view(Mb, 128, Kb, 128)
    scale = tiles.abs().amax((1, 3)) / E4M3_MAX
    codes = (tiles / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(Mb * 128, Kb * 128)[:M, :K]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


def _rows(T, K, g):
    """Rows as a block sees them: normal, a few channels far larger than the rest, tokens of different size."""
    x = torch.randn(T, K, generator=g, device=DEV)
    x *= 1 + 20 * (torch.rand(K, generator=g, device=DEV) < 0.01)
    return x.mul_(0.5 + torch.rand(T, 1, generator=g, device=DEV))


def _activations(T, K, g):
    """8-bit activations [T][K] with scales [ceil(K / 128)][T]."""
    Kb = -(-K // 128)
    full = torch.zeros(T, Kb * 128, device=DEV)
    full[:, :K] = _rows(T, K, g) * 0.5
    blocks = full.view(T, Kb, 128)
    scale = blocks.abs().amax(-1) / E4M3_MAX
    codes = (blocks / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, Kb * 128)[:, :K]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale.t().contiguous()


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": case}
    T = case["T"]
    if case["op"] == "norm":
        H = case["H"]
        s["x"] = _rows(T, H, g).to(_TYPES[case["x"]])
        s["res"] = (4 * _rows(T, H, g)).to(_TYPES[case["res"]])
        s["post_w"] = 1 + 0.2 * torch.randn(H, generator=g, device=DEV) if case["post"] else None
        s["pre_w"] = 1 + 0.2 * torch.randn(H, generator=g, device=DEV)
        s["gate"] = None
        if case["gate"] != "none":
            rows = T if case["gate"] == "full" else 1
            s["gate"] = torch.sigmoid(torch.randn(rows, H, generator=g, device=DEV)).to(torch.bfloat16)
        s["scale"], s["eps"] = 0.75, 1e-6
    elif case["op"] == "encode":
        s["x"] = _rows(T, case["K"], g).to(_TYPES[case["x"]])
    else:
        s["x"], s["xs"] = _activations(T, case["K"], g)
        if case["op"] == "gemm":
            s["w"], s["ws"] = _weight(case["M"], case["K"], g)
        else:
            s["wg"], s["wgs"] = _weight(case["I"], case["K"], g)
            s["wu"], s["wus"] = _weight(case["I"], case["K"], g)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # what a program keeps from step to step: output buffers
        import block_quantized_decode_nvfp4_gb300 as bqd
        s["bqd"] = bqd
        s["types"] = {"f32": bqd.BQD_F32, "bf16": bqd.BQD_BF16, "e4m3": bqd.BQD_E4M3}
        T, op = case["T"], case["op"]

        def out(kind, n):
            dt = torch.float8_e4m3fn if kind == "e4m3" else _TYPES[kind]
            return torch.empty(T, n, dtype=dt, device=DEV)

        def scales(kind, n):
            return torch.empty(-(-n // 128), T, device=DEV) if kind == "e4m3" else None

        if op == "norm":
            s["res_out"] = torch.empty_like(s["res"])
            s["y"], s["ys"] = out(case["y"], case["H"]), scales(case["y"], case["H"])
        elif op == "encode":
            s["y"], s["ys"] = out("e4m3", case["K"]), scales("e4m3", case["K"])
        elif op == "gemm":
            s["y"] = out(case["y"], case["M"])
        else:
            s["y"], s["ys"] = out(case["h"], case["I"]), scales(case["h"], case["I"])
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    return _RUN[s["case"]["op"], bool(own)](s)


def _norm_own(s):
    c, b, t = s["case"], s["bqd"], s["types"]
    H = c["H"]
    b.residual_norm(s["x"], t[c["x"]], H, s["post_w"], s["gate"], b.BQD_BF16, H if c["gate"] == "full" else 0,
                    s["scale"], s["res"], s["res_out"], t[c["res"]], s["pre_w"], s["eps"], s["y"], t[c["y"]], s["ys"],
                    H, c["T"])
    return {"res": s["res_out"], "y": s["y"], "scales": s["ys"]} if s["ys"] is not None else \
        {"res": s["res_out"], "y": s["y"]}


def _encode_own(s):
    c = s["case"]
    s["bqd"].fp8_x_encode(s["x"], s["types"][c["x"]], c["K"], s["y"], s["ys"], c["K"], c["T"])
    return {"y": s["y"], "scales": s["ys"]}


def _gemm_own(s):
    c = s["case"]
    s["bqd"].fp8_b128_gemm(s["w"], s["ws"], s["x"], s["xs"], s["y"], s["types"][c["y"]], c["M"], c["K"], c["T"])
    return {"y": s["y"]}


def _ffn_own(s):
    c = s["case"]
    s["bqd"].fp8_b128_gemm_silu_mul(s["wg"], s["wgs"], s["wu"], s["wus"], s["x"], s["xs"], s["y"], s["types"][c["h"]],
                                    s["ys"], c["I"], c["K"], c["T"])
    return {"h": s["y"], "scales": s["ys"]} if s["ys"] is not None else {"h": s["y"]}


def _blocks(x):
    """[T][K] as [T][ceil(K / 128)][128], zeros past K."""
    T, K = x.shape
    pad = -K % 128
    if pad:
        x = torch.cat([x, torch.zeros(T, pad, dtype=x.dtype, device=x.device)], 1)
    return x.view(T, -1, 128)


def _to_codes(x):
    """E4M3 codes [T][K] and scales [ceil(K / 128)][T] of fp32 rows."""
    T, K = x.shape
    b = _blocks(x)
    s = (b.abs().amax(-1) / E4M3_MAX).clamp(min=TINY)
    q = (b / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(T, -1)[:, :K]
    return q.to(torch.float8_e4m3fn), s.t().contiguous()


def _norm_plain(s):
    c = s["case"]
    z = s["x"].float()
    if c["post"]:
        z = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + s["eps"]) * s["post_w"]
    if s["gate"] is not None:
        z = z * s["gate"].float()
    r = s["res"].float() + s["scale"] * z
    y = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + s["eps"]) * s["pre_w"]
    res = r.to(s["res"].dtype)
    if c["y"] == "bf16":
        return {"res": res, "y": y.to(torch.bfloat16)}
    codes, scales = _to_codes(y)
    return {"res": res, "y": codes, "scales": scales}


def _encode_plain(s):
    codes, scales = _to_codes(s["x"].float())
    return {"y": codes, "scales": scales}


def _value_x(x, xs):
    K = x.shape[1]
    return x.float() * xs.t().repeat_interleave(128, 1)[:, :K]


def _value_w(w, ws):
    M, K = w.shape
    return w.float() * ws.repeat_interleave(128, 0)[:M].repeat_interleave(128, 1)[:, :K]


def _gemm_plain(s):
    y = torch.matmul(_value_x(s["x"], s["xs"]), _value_w(s["w"], s["ws"]).t())
    return {"y": y.to(_TYPES[s["case"]["y"]])}


def _ffn_plain(s):
    x = _value_x(s["x"], s["xs"])
    g = torch.matmul(x, _value_w(s["wg"], s["wgs"]).t())
    u = torch.matmul(x, _value_w(s["wu"], s["wus"]).t())
    h = g / (1 + torch.exp(-g)) * u
    kind = s["case"]["h"]
    if kind != "e4m3":
        return {"h": h.to(_TYPES[kind])}
    codes, scales = _to_codes(h)
    return {"h": codes, "scales": scales}


_RUN = {("norm", True): _norm_own, ("norm", False): _norm_plain,
        ("encode", True): _encode_own, ("encode", False): _encode_plain,
        ("gemm", True): _gemm_own, ("gemm", False): _gemm_plain,
        ("ffn", True): _ffn_own, ("ffn", False): _ffn_plain}


# ---------------------------------------------------------------- what a pass cannot do without
_SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}


def work(case):
    T, op = case["T"], case["op"]
    if op == "norm":
        H = case["H"]
        per = _SIZE[case["x"]] + 2 * _SIZE[case["res"]] + _SIZE[case["y"]] + (2 if case["gate"] == "full" else 0)
        n = T * H * per + 4 * H * (2 if case["post"] else 1) + (2 * H if case["gate"] == "row" else 0)
        n += 4 * T * -(-H // 128) if case["y"] == "e4m3" else 0
        return {"bytes": n, "flops": T * H * (11 if case["post"] else 7)}
    K = case["K"]
    Kb = -(-K // 128)
    if op == "encode":
        return {"bytes": T * K * (_SIZE[case["x"]] + 1) + 4 * T * Kb, "flops": 2 * T * K}
    x = T * K + 4 * T * Kb
    if op == "gemm":
        M = case["M"]
        return {"bytes": x + M * K + 4 * -(-M // 128) * Kb + T * M * _SIZE[case["y"]], "flops": 2 * T * M * K}
    I = case["I"]
    n = x + 2 * (I * K + 4 * -(-I // 128) * Kb) + T * I * _SIZE[case["h"]]
    n += 4 * T * -(-I // 128) if case["h"] == "e4m3" else 0
    return {"bytes": n, "flops": 4 * T * I * K}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_codes(v):
    """What the codes stand for before their rounding, and the scales: v [T][K] fp64, 128 columns at a time."""
    T, K = v.shape
    q, s = torch.empty_like(v), torch.empty(-(-K // 128), T, dtype=torch.float64, device=v.device)
    for j in range(0, K, 128):
        part = v[:, j:j + 128]
        s[j // 128] = torch.clamp(part.abs().max(1).values / E4M3_MAX, min=TINY)
        q[:, j:j + 128] = part / s[j // 128][:, None]
    return q, s


def _exact_product(x, xs, w, ws):
    """[T][M] fp64: 128 k and 128 rows of the weights at a time, each with its own scales."""
    T, K = x.shape
    M = w.shape[0]
    a = x.double()
    for j in range(0, K, 128):
        a[:, j:j + 128] *= xs[j // 128].double()[:, None]
    y = torch.empty(T, M, dtype=torch.float64, device=x.device)
    for i in range(0, M, 2048):
        b = w[i:i + 2048].double()
        for n in range(0, b.shape[0], 128):
            for j in range(0, K, 128):
                b[n:n + 128, j:j + 128] *= ws[(i + n) // 128, j // 128].double()
        y[:, i:i + 2048] = a @ b.t()
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "norm":
        z = s["x"].double()
        if s["post_w"] is not None:
            z = z / torch.sqrt(z.pow(2).sum(1, keepdim=True) / case["H"] + s["eps"]) * s["post_w"].double()
        if s["gate"] is not None:
            z = z * s["gate"].double()
        r = s["res"].double() + s["scale"] * z
        y = r / torch.sqrt(r.pow(2).sum(1, keepdim=True) / case["H"] + s["eps"]) * s["pre_w"].double()
        if case["y"] == "bf16":
            return {"res": r, "y": y}
        q, sc = _exact_codes(y)
        return {"res": r, "y": q, "scales": sc}
    if op == "encode":
        q, sc = _exact_codes(s["x"].double())
        return {"y": q, "scales": sc}
    if op == "gemm":
        return {"y": _exact_product(s["x"], s["xs"], s["w"], s["ws"])}
    g = _exact_product(s["x"], s["xs"], s["wg"], s["wgs"])
    u = _exact_product(s["x"], s["xs"], s["wu"], s["wus"])
    h = g * torch.sigmoid(g) * u
    if case["h"] != "e4m3":
        return {"h": h}
    q, sc = _exact_codes(h)
    return {"h": q, "scales": sc}
