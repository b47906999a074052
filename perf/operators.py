"""What the int8 scaled-product operators compute, on which sizes, and what they cannot do without.

Three operators: the per-row int8 quantization (optionally gathering rows for the experts, optionally
with the SiLU gate between an expert's two products), the int8 product with a scale per token and per
channel (from int8 rows, or from the unquantized rows in one call), and the same product grouped by
expert over ragged row groups.

Codes are int8 row-major matrices whose rows start 16 bytes apart or a multiple of that, scales fp32.
The plain forms are elementary torch operations in 32 bits. Their integer sums are exact: every product
is a whole number below 2^14, and with the codes drawn here (normal, standard deviation 32) a sum over
K <= 13824 has a standard deviation of 32 * 32 * sqrt(13824) = 1.2e5, far below 2^24.
"""
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decoded token before a 4096-wide layer
        dict(name="quantize 1x4096", op="quantize", M=1, K=4096, x="bf16", gate=False, rows=0),
        # a prefill batch's tokens, taken in the experts' order (each token goes to two experts)
        dict(name="quantize gather 16384x4096", op="quantize", M=16384, K=4096, x="bf16", gate=False, rows=8192),
        # gate and up halves of one product's output, gated and quantized for the down product
        dict(name="quantize gated 4096x11008", op="quantize", M=4096, K=11008, x="bf16", gate=True, rows=0),
        # one decoded token through an attention projection
        dict(name="linear 1x4096x4096", op="linear", M=1, N=4096, K=4096, x="bf16", y="bf16", bias=False),
        # a small decoding batch through an up projection
        dict(name="linear 16x11008x4096", op="linear", M=16, N=11008, K=4096, x="bf16", y="bf16", bias=False),
        # a chunk of a prompt at odd sizes, with a bias
        dict(name="gemm 333x5120x5111", op="gemm", M=333, N=5120, K=5111, y="fp16", bias=True),
        # a prompt through a down projection
        dict(name="gemm 2048x4096x11008", op="gemm", M=2048, N=4096, K=11008, y="bf16", bias=False),
        # the largest prefill batch through an up projection
        dict(name="gemm 8192x13824x5120", op="gemm", M=8192, N=13824, K=5120, y="bf16", bias=False),
        # decoding: 8 tokens to two of 16 experts each
        dict(name="grouped 16e 16x4096x2048", op="grouped", E=16, M=16, N=4096, K=2048, skew=0.5, y="bf16", bias=False),
        # many small experts, a ragged prefill, fp32 outputs
        dict(name="grouped 64e 4100x2048x2048", op="grouped", E=64, M=4100, N=2048, K=2048, skew=0.5, y="fp32", bias=True),
        # few large experts, the largest prefill
        dict(name="grouped 8e 16384x11008x4096", op="grouped", E=8, M=16384, N=11008, K=4096, skew=0.3, y="bf16", bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "gemm", "grouped"])
    if op == "quantize":
        gate = rng.random() < 0.4
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 100, 13824), x=rng.choice(["bf16", "fp16", "fp32"]),
                    gate=gate, rows=0 if gate or rng.random() < 0.5 else _log(rng, 1, 8192))
    c = dict(op=op, N=_log(rng, 256, 13824), K=_log(rng, 100, 11008), y=rng.choice(["bf16", "fp16", "fp32"]),
             bias=rng.random() < 0.5)
    if op == "linear":
        c |= dict(M=_log(rng, 1, 512), x=rng.choice(["bf16", "fp16", "fp32"]))
    elif op == "gemm":
        c |= dict(M=_log(rng, 1, 8192))
    else:
        c |= dict(E=_log(rng, 2, 64), M=_log(rng, 4, 8192), N=_log(rng, 256, 4096), K=_log(rng, 100, 4096),
                  skew=round(rng.random(), 2))
    return c


# ---------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------

def _codes(shape, g):
    """int8 codes as absmax quantization leaves them, in rows that start on 16-byte boundaries."""
    K = shape[-1]
    buf = torch.empty(*shape[:-1], (K + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    for part in (buf.view(-1, buf.shape[-1]).split(1 << 15)):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").mul_(32).round_().clamp_(-127, 127))
    return buf[..., :K]


def _scales(shape, g):
    return torch.rand(shape, generator=g, device="cuda") * 2e-3 + 1e-4


def _rows(M, K, kind, g):
    """Activations: normal, with a few wide channels and tokens of differing size."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x[:, ::97] *= 8
    x *= torch.rand(M, 1, generator=g, device="cuda") * 2 + 0.1
    return x.to(_TYPES[kind])


def _counts(E, M, skew, seed):
    """Rows of each expert: proportional to 1 + skew * u with u in (-1, 1), one expert in eight empty."""
    r = torch.Generator().manual_seed(seed)
    w = 1 + skew * (2 * torch.rand(E, generator=r) - 1)
    if E >= 8:
        w[torch.randperm(E, generator=r)[: E // 8]] = 0
    edges = (torch.cumsum(w, 0) / w.sum() * M).round().to(torch.int64)
    edges[-1] = M
    return torch.diff(edges, prepend=torch.zeros(1, dtype=torch.int64)).clamp_(min=0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, M, K = case["op"], case["M"], case["K"]
    s = dict(op=op, layer=None)
    if op == "quantize":
        n = case["rows"] or M
        if case["gate"]:
            both = torch.cat([_rows(n, K, case["x"], g), _rows(n, K, case["x"], g)], 1)  # gate | up
            s |= dict(gate=both[:, :K], x=both[:, K:])
        else:
            s |= dict(gate=None, x=_rows(n, K, case["x"], g))
        s["rows"] = torch.randint(0, n, (M,), generator=g, device="cuda", dtype=torch.int32) if case["rows"] else None
        return s
    lead = (case["E"],) if op == "grouped" else ()
    s |= dict(w=_codes((*lead, case["N"], K), g), sw=_scales((*lead, case["N"]), g), y=_TYPES[case["y"]],
              bias=torch.randn((*lead, case["N"]), generator=g, device="cuda") if case["bias"] else None)
    if op == "linear":
        s["x"] = _rows(M, K, case["x"], g)
        return s
    s |= dict(q=_codes((M, K), g), sa=_scales((M,), g))
    if op == "grouped":
        counts = _counts(case["E"], M, case["skew"], seed)
        s["most"] = int(counts.max())
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
    return s


# ---------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------

def _plain_quantize(x, gate, rows):
    if rows is not None:
        x = x[rows]
        gate = None if gate is None else gate[rows]
    v = x.float()
    if gate is not None:
        g = gate.float()
        v = v * (g / (1 + torch.exp(-g)))
    gamma = v.abs().amax(1)
    fine = torch.isfinite(gamma)
    some = fine & (gamma >= 2.0 ** -100)
    s = torch.where(some, 127 / gamma, torch.zeros_like(gamma))
    q = torch.where(some[:, None], torch.round(v * s[:, None]), torch.zeros_like(v)).to(torch.int8)
    scale = torch.where(some, gamma / 127, torch.where(fine, torch.zeros_like(gamma), torch.full_like(gamma, float("nan"))))
    return q, scale


def _plain_gemm(q, sa, w, sw, bias, kind):
    y = torch.matmul(q.float(), w.float().transpose(-1, -2)) * (sa[..., :, None] * sw[..., None, :])
    if bias is not None:
        y = y + bias[..., None, :]
    return y.to(kind)


def _plain_grouped(q, sa, w, sw, bias, offsets, most, kind):
    first, row = offsets[:-1].long(), torch.arange(q.shape[0], device=q.device)
    slot = (first[:, None] + torch.arange(most, device=q.device)).clamp(max=q.shape[0] - 1)  # [E, most]
    y = _plain_gemm(q[slot], sa[slot], w, sw, bias, kind)
    expert = torch.searchsorted(offsets[1:].long(), row, right=True)
    return y[expert, row - first[expert]]


def run(state):
    op = state["op"]
    if own:
        from bit_weight_quantization_b200 import bq
        if op == "quantize":
            return bq.scaled_quantize(state["x"], gate=state["gate"], rows=state["rows"])
        layer = state["layer"]
        if layer is None:  # the program's handle on its weights
            layer = state["layer"] = bq.ScaledLinear(state["w"], state["sw"], state["bias"])
        if op == "linear":
            return layer.linear(state["x"], dtype=state["y"])
        if op == "gemm":
            return layer.gemm(state["q"], state["sa"], dtype=state["y"])
        return layer.gemm_grouped(state["q"], state["sa"], state["offsets"], dtype=state["y"])
    if op == "quantize":
        return _plain_quantize(state["x"], state["gate"], state["rows"])
    if op == "linear":
        q, sa = _plain_quantize(state["x"], None, None)
        return _plain_gemm(q, sa, state["w"], state["sw"], state["bias"], state["y"])
    if op == "gemm":
        return _plain_gemm(state["q"], state["sa"], state["w"], state["sw"], state["bias"], state["y"])
    return _plain_grouped(state["q"], state["sa"], state["w"], state["sw"], state["bias"], state["offsets"],
                          state["most"], state["y"])


# ---------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------------

def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    if op == "quantize":
        read = min(M, case["rows"] or M) * K * _SIZE[case["x"]] * (2 if case["gate"] else 1)
        return dict(bytes=read + M * K + 4 * M + (4 * M if case["rows"] else 0), flops=(8 if case["gate"] else 3) * M * K)
    N = case["N"]
    out = M * N * _SIZE[case["y"]]
    used = 1
    if op == "grouped":  # the experts that have rows; which ones goes by the seed, how many hardly does
        used = int((_counts(case["E"], M, case["skew"], 0) > 0).sum())
    weights = used * (N * K + 4 * N * (2 if case["bias"] else 1))
    tokens = M * K * (_SIZE[case["x"]] if op == "linear" else 1) + (0 if op == "linear" else 4 * M)
    return dict(bytes=weights + tokens + out, flops=2 * M * N * K)


# ---------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------

def exact(case, seed):
    """The products in 64 bits. The codes are whole numbers that the definition fixes through two roundings
    to 32 bits (127 / gamma and its product with x): they are made so here too, and the rest in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("quantize", "linear"):
        x = s["x"] if s.get("rows") is None else s["x"].index_select(0, s["rows"])
        if s.get("gate") is not None:
            gate = s["gate"].double()
            v = x.double() * gate / (1 + torch.exp(-gate))
            return [None, v.abs().max(1).values / 127]  # a code next to a tie hangs on the last bit of exp
        x = x.double()
        gamma = x.abs().max(1).values
        inverse = (127 / gamma).float().double()  # correctly rounded: 127 / gamma in 64 bits is never next to a tie
        q = torch.round((x * inverse[:, None]).float().double())
        if op == "quantize":
            return [q.to(torch.int8), gamma / 127]
        sa = gamma / 127
    else:
        q, sa = s["q"].double(), s["sa"].double()
    bias = None if s["bias"] is None else s["bias"].double()

    def product(rows, scale, w, sw, b):
        out = torch.empty(rows.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
        for n in range(0, w.shape[0], 2048):
            out[:, n:n + 2048] = rows @ w[n:n + 2048].double().t()
        out *= scale[:, None] * sw.double()
        return out if b is None else out + b

    if op != "grouped":
        return product(q, sa, s["w"], s["sw"], bias)
    y = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
    edges = s["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(edges, edges[1:])):
        if hi > lo:
            y[lo:hi] = product(q[lo:hi], sa[lo:hi], s["w"][e], s["sw"][e], None if bias is None else bias[e])
    return y
