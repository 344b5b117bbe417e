"""The 8-bit feed-forward operators as they are measured: cases, inputs, plain forms, exact values.

A case names one of five operators:

  quant_int8    x bf16 [M, K] -> int8 codes and one FP32 scale per row
  gemm_int8     C = (qa qb^T) scaled per token and per channel, int8 x int8 with exact sums
  int8_gated    h = silu(gate) * up, both projections from one int8 weight of 2N rows
  fp8_gated     the same from E4M3 codes with 1x128 activation and 128x128 weight scales
  train         forward and backward of the FP8 gated projections from bf16 x, w and dh

With ``own`` false, run() computes them in plain torch operations; with ``own`` true it
calls the library.  A stacked weight has the gate's N rows first, then the up
projection's.  Definitions (all in real numbers but for the roundings named):

  int8 rows     s = RN32(amax / 127), r = RN32(127 / amax), q = round-half-even(x r)
  E4M3 tiles    s = RN32(amax / 448) (power of two: the next one up), q = E4M3(RN32(x / s))
  gated         h = g u / (1 + exp(-g))
  gated bwd     from g, u rounded to bf16: du = dh silu(g), dg = dh u silu'(g), both rounded
                to bf16 and quantized (1x128 along N for dx, along the tokens for dw);
                x is quantized along K for h and along the tokens for dw
"""
import math

import torch

own = False

KINDS = ("quant_int8", "gemm_int8", "int8_gated", "fp8_gated", "train")


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one new token's activations before an int8 product (latency)
        {"name": "quant_int8 1x7168", "op": "quant_int8", "M": 1, "N": 0, "K": 7168},
        # a prefill batch's activations
        {"name": "quant_int8 16384x7168", "op": "quant_int8", "M": 16384, "N": 0, "K": 7168},
        # the down projection of one expert for one token
        {"name": "gemm_int8 1x7168x2048", "op": "gemm_int8", "M": 1, "N": 7168, "K": 2048, "fp32": False},
        # a decode batch through a square projection
        {"name": "gemm_int8 64x7168x7168", "op": "gemm_int8", "M": 64, "N": 7168, "K": 7168, "fp32": False},
        # odd and ragged sizes, FP32 output
        {"name": "gemm_int8 1001x2047x1499 fp32", "op": "gemm_int8", "M": 1001, "N": 2047, "K": 1499, "fp32": True},
        # the dense workload's product in int8
        {"name": "gemm_int8 4096x7168x7168", "op": "gemm_int8", "M": 4096, "N": 7168, "K": 7168, "fp32": False},
        # gate and up projections of one expert for one token
        {"name": "int8_gated 1x2048x7168", "op": "int8_gated", "M": 1, "N": 2048, "K": 7168},
        # the same for a prefill batch
        {"name": "int8_gated 4096x2048x7168", "op": "int8_gated", "M": 4096, "N": 2048, "K": 7168},
        # a decode batch of one expert, FP8
        {"name": "fp8_gated 16x2048x7168", "op": "fp8_gated", "M": 16, "N": 2048, "K": 7168, "pow2": False},
        # a prefill batch of one expert, FP8
        {"name": "fp8_gated 8192x2048x7168", "op": "fp8_gated", "M": 8192, "N": 2048, "K": 7168, "pow2": False},
        # a small training step with a ragged number of tokens
        {"name": "train 200x256x384", "op": "train", "M": 200, "N": 256, "K": 384, "pow2": False},
        # a training step of one expert
        {"name": "train 8192x2048x7168 pow2", "op": "train", "M": 8192, "N": 2048, "K": 7168, "pow2": True},
    ]


MOST_FLOPS = 2.0 * 4096 * 7168 * 7168      # a drawn product's multiply-adds, at most


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(KINDS)
    M = _log_int(rng, 1, 16384)
    if op == "quant_int8":
        return {"op": op, "M": M, "N": 0, "K": _log_int(rng, 64, 8192)}
    if op in ("gemm_int8", "int8_gated"):
        N, K = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
    else:
        N, K = 128 * _log_int(rng, 1, 32), 128 * _log_int(rng, 1, 64)
    per_row = 2.0 * N * K * {"gemm_int8": 1, "int8_gated": 2, "fp8_gated": 2, "train": 6}[op]
    M = max(1, min(M, int(MOST_FLOPS / per_row)))
    case = {"op": op, "M": M, "N": N, "K": K}
    if op == "gemm_int8":
        case["fp32"] = rng.random() < 0.3
    if op in ("fp8_gated", "train"):
        case["pow2"] = rng.random() < 0.5
    return case


def work(case):
    """Bytes each input is read and each output written once; multiply-adds count two."""
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    if op == "quant_int8":
        return {"bytes": 3 * M * K + 4 * M, "flops": 2 * M * K}
    if op == "gemm_int8":
        return {"bytes": (M + N) * K + 4 * (M + N) + (4 if case["fp32"] else 2) * M * N, "flops": 2 * M * N * K}
    if op == "int8_gated":
        return {"bytes": (M + 2 * N) * K + 4 * (M + 2 * N) + 2 * M * N, "flops": 4 * M * N * K}
    if op == "fp8_gated":
        return {"bytes": (M + 2 * N) * K + 4 * M * (K // 128) + 4 * (N // 64) * (K // 128) + 2 * M * N,
                "flops": 4 * M * N * K}
    return {"bytes": 4 * M * K + 8 * N * K + 4 * M * N, "flops": 12 * M * N * K}


# ----------------------------------------------------------------------------------- inputs

def _normal(g, shape, std):
    return torch.randn(shape, generator=g, device="cuda") * std


def _activations(g, M, K):
    """N(0, 1) activations with a thousandth of outliers a hundred times larger."""
    x = _normal(g, (M, K), 1.0)
    x.mul_(1.0 + 99.0 * (torch.rand((M, K), generator=g, device="cuda") < 0.001))
    return x.to(torch.bfloat16)


def _pitched(t):
    """`t` with rows that start on 16 bytes, as the quantizer lays out codes of any K."""
    M, K = t.shape
    pitch = -(-K // 16) * 16
    buf = torch.zeros((M, pitch), dtype=t.dtype, device=t.device)
    buf[:, :K] = t
    return buf[:, :K]


def prepare(case, seed):
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    st = dict(case)
    x = _activations(g, M, K)
    if op == "quant_int8":
        st["x"] = x
    elif op in ("gemm_int8", "int8_gated"):
        rows = N if op == "gemm_int8" else 2 * N
        w = _normal(g, (rows, K), 1.0 / math.sqrt(K)).to(torch.bfloat16)
        q, st["sa"] = _rows_int8(x)
        st["qa"] = _pitched(q)
        q, st["sw"] = _rows_int8(w)
        st["qw"] = _pitched(q)
    else:
        w = _normal(g, (2 * N, K), 1.0 / math.sqrt(K)).to(torch.bfloat16)
        if op == "fp8_gated":
            q, s = _tiles(x, case["pow2"])
            st["qa"], st["sa"] = q.view(torch.uint8), s.t().contiguous()
            q, st["sw"] = _blocks(w, case["pow2"])
            st["qw"] = q.view(torch.uint8)
        else:
            st["x"] = x.requires_grad_(True)
            st["w"] = w.requires_grad_(True)
            st["dh"] = _normal(g, (M, N), 1e-3).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------------------ plain forms

def _rows_int8(x):
    a = x.abs().amax(dim=1).float()
    c = torch.full_like(a, 127.0)
    s = torch.where(a > 0, a / c, torch.ones_like(a))
    r = torch.where(a > 0, c / a, torch.zeros_like(a))
    # the product of a bf16 and an FP32 number is exact in 64 bits: one rounding
    q = torch.round(x.double() * r.double()[:, None]).to(torch.int8)
    return q, s


def _scale448(a, pow2):
    s = torch.where(a > 0, a / torch.full_like(a, 448.0), torch.ones_like(a))
    if pow2:
        m, e = torch.frexp(s)                       # s = m 2^e, m in [0.5, 1)
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    return s


def _tiles(x, pow2):
    """1x128 tiles along the last dimension (the last one may be short): E4M3 [M, K], scales [M, tiles]."""
    M, K = x.shape
    T = -(-K // 128)
    p = torch.nn.functional.pad(x.float(), (0, T * 128 - K)).view(M, T, 128)
    s = _scale448(p.abs().amax(dim=2), pow2)
    q = (p / s[:, :, None]).view(M, T * 128)[:, :K].to(torch.float8_e4m3fn)
    return q, s


def _blocks(w, pow2):
    """128x128 blocks: E4M3 [R, K], scales [R / 128, K / 128]."""
    R, K = w.shape
    b = w.float().view(R // 128, 128, K // 128, 128)
    s = _scale448(b.abs().amax(dim=(1, 3)), pow2)
    return (b / s[:, None, :, None]).view(R, K).to(torch.float8_e4m3fn), s


def _tile_values(q, s):
    return q.float() * s.repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _block_values(q, s):
    return q.float() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)


def _gate(g, u):
    return g * u / (1 + torch.exp(-g))


def _plain_train(x, w, dh, pow2):
    N = dh.shape[1]
    wv = _block_values(*_blocks(w, pow2))
    gu = _tile_values(*_tiles(x, pow2)) @ wv.t()
    h = _gate(gu[:, :N], gu[:, N:]).to(torch.bfloat16)
    gu = gu.to(torch.bfloat16).float()
    g, u, d = gu[:, :N], gu[:, N:], dh.float()
    sg = 1 / (1 + torch.exp(-g))
    dgu = torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], 1).to(torch.bfloat16)
    dx = _tile_values(*_tiles(dgu, pow2)) @ wv
    dw = _tile_values(*_tiles(dgu.t(), pow2)) @ _tile_values(*_tiles(x.t(), pow2)).t()
    return h, dx.to(torch.bfloat16), dw.to(torch.bfloat16)


def _plain(st):
    op, N = st["op"], st["N"]
    if op == "quant_int8":
        return _rows_int8(st["x"])
    if op == "train":
        return _plain_train(st["x"].detach(), st["w"].detach(), st["dh"], st["pow2"])
    if op == "fp8_gated":
        a = _tile_values(st["qa"].view(torch.float8_e4m3fn), st["sa"].t())
        gu = a @ _block_values(st["qw"].view(torch.float8_e4m3fn), st["sw"]).t()
        return _gate(gu[:, :N], gu[:, N:]).to(torch.bfloat16)
    c = (st["qa"].float() @ st["qw"].float().t()) * st["sa"][:, None] * st["sw"]
    if op == "gemm_int8":
        return c if st["fp32"] else c.to(torch.bfloat16)
    return _gate(c[:, :N], c[:, N:]).to(torch.bfloat16)


def run(state):
    if not own:
        return _plain(state)
    import fp8_fine_grained_weight_b200 as fq
    from fp8_fine_grained_weight_b200.linear import fp8_gated_linear
    op = state["op"]
    if op == "quant_int8":
        return fq.quant_int8_rowwise(state["x"])
    if op == "gemm_int8":
        return fq.gemm_int8(state["qa"], state["sa"], state["qw"], state["sw"],
                            out_dtype=torch.float32 if state["fp32"] else torch.bfloat16)
    if op == "int8_gated":
        return fq.gemm_int8_gated(state["qa"], state["sa"], state["qw"], state["sw"])
    if op == "fp8_gated":
        return fq.gemm_blockscaled_gated(state["qa"], state["sa"], state["qw"], state["sw"])
    h = fp8_gated_linear(state["x"], state["w"], state["pow2"])
    dx, dw = torch.autograd.grad(h, (state["x"], state["w"]), state["dh"])
    return h.detach(), dx, dw


# ------------------------------------------------------------------------------ exact values

def _e4m3_64(v):
    """Nearest E4M3 value of each 64-bit number, ties to even, 448 at most."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -12)))
    e = torch.where(v.abs() < torch.exp2(e), e - 1, torch.where(v.abs() >= torch.exp2(e + 1), e + 1, e))
    step = torch.exp2(e.clamp_min(-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _dequantized_64(x, tile_rows, tile_cols, pow2):
    """x quantized in tile_rows x tile_cols tiles and read back, in 64 bits.  The FP32
    roundings of the scale and of the quotient are the definition's."""
    R, C = x.shape
    pr, pc = -R % tile_rows, -C % tile_cols
    t = torch.zeros((R + pr, C + pc), dtype=torch.float64, device=x.device)
    t[:R, :C] = x.double()
    t = t.view((R + pr) // tile_rows, tile_rows, (C + pc) // tile_cols, tile_cols)
    amax = t.abs().amax(dim=3, keepdim=True).amax(dim=1, keepdim=True)
    s = (amax / 448.0).float().double()
    if pow2:
        up = torch.exp2(torch.ceil(torch.log2(s.clamp_min(1e-300))))
        up = torch.where(up / 2 >= s, up / 2, torch.where(up < s, up * 2, up))
        s = up
    s = torch.where(amax == 0, torch.ones_like(s), s)
    v = _e4m3_64((t / s).float().double()) * s
    return v.reshape(R + pr, C + pc)[:R, :C]


def _sigmoid_64(g):
    return torch.special.expit(g)


def exact(case, seed):
    st = prepare(case, seed)
    op, N = case["op"], case["N"]
    if op == "quant_int8":
        x = st["x"].double()
        amax = x.abs().max(dim=1).values
        zero = amax == 0
        scale = torch.where(zero, 1.0, (amax / 127.0))
        r = torch.where(zero, 0.0, (127.0 / amax).float().double())
        return torch.round(x * r.unsqueeze(1)).to(torch.int8), scale
    if op in ("gemm_int8", "int8_gated"):
        acc = torch.matmul(st["qa"].double(), st["qw"].double().transpose(0, 1))
        acc = acc * st["sa"].double().unsqueeze(1) * st["sw"].double().unsqueeze(0)
        if op == "gemm_int8":
            return acc
        return acc[:, :N] * _sigmoid_64(acc[:, :N]) * acc[:, N:]
    if op == "fp8_gated":
        tiles, blocks = case["K"] // 128, case["N"] // 64
        a = st["qa"].view(torch.float8_e4m3fn).double().view(-1, tiles, 128)
        a = (a * st["sa"].double().t().unsqueeze(2)).view(-1, case["K"])
        w = st["qw"].view(torch.float8_e4m3fn).double().view(blocks, 128, tiles, 128)
        w = (w * st["sw"].double().view(blocks, 1, tiles, 1)).view(-1, case["K"])
        p = torch.matmul(a, w.transpose(0, 1))
        return p[:, :N] * _sigmoid_64(p[:, :N]) * p[:, N:]
    pow2 = case["pow2"]
    x, w = st["x"].detach(), st["w"].detach()
    w64 = _dequantized_64(w, 128, 128, pow2)
    p = torch.matmul(_dequantized_64(x, 1, 128, pow2), w64.transpose(0, 1))
    h = p[:, :N] * _sigmoid_64(p[:, :N]) * p[:, N:]
    p = p.to(torch.bfloat16).double()          # what the forward pass keeps
    g, u, dh = p[:, :N], p[:, N:], st["dh"].double()
    sg = _sigmoid_64(g)
    d = torch.empty_like(p)
    d[:, :N] = dh * u * (sg + g * sg * (1.0 - sg))
    d[:, N:] = dh * g * sg
    d = d.to(torch.bfloat16)                   # what is quantized
    dx = torch.matmul(_dequantized_64(d, 1, 128, pow2), w64)
    del w64
    dw = torch.matmul(_dequantized_64(d, 128, 1, pow2).transpose(0, 1), _dequantized_64(x, 128, 1, pow2))
    return h, dx, dw
