"""Workloads of the 4-bit weight products and of the mixture-of-experts token
operators: inputs, plain forms and the library's calls.

Operators (case["op"]):

* ``int4_mm``: C = bf16(x . dequant(B)^T [+ bias]), B 4-bit codes with a bf16
  scale (and optionally a zero point) per group of G weights of a row;
* ``grouped_int4_mm``: the same for every expert's rows of a sorted batch;
* ``moe_sort``: expert ids of every token -> offsets, order and slots of the
  rows sorted by expert;
* ``moe_permute`` (direction forward: bf16 rows or quantized rows; backward:
  the sum of a token's row gradients);
* ``moe_unpermute`` (forward: weighted sum of a token's rows; backward: the
  rows' and the weights' gradients).

The plain forms compute in fp32 with elementary torch operations and round
once.  Sizes are those of Qwen3 decoder layers (dense 8B and 32B, 30B-A3B
experts), as in ``quantized_linear_gemm_b200/inputs.py``, or generic.
"""

import math

import torch

own = False

HIDDEN, INTER, EXPERTS, TOP_K = 2048, 768, 128, 8   # Qwen3-30B-A3B

# work of the largest listed product and largest listed token case
_MAX_FLOPS = 2 * 2048 * 24576 * 4096
_MAX_ROWS_BYTES = 4096 * HIDDEN * 2 * (TOP_K * 2 + 1)


def listed():
    return [
        # one token of a decode step: the QKV projection of an 8B layer; latency counts
        dict(name="int4_decode_m1", op="int4_mm", M=1, N=6144, K=4096, G=128, zeros=False, bias=False),
        # a small decode batch on the widest 8B linear: the weight stream decides
        dict(name="int4_decode_m8", op="int4_mm", M=8, N=24576, K=4096, G=128, zeros=True, bias=False),
        # an odd decode batch on the longest rows (32B down projection), finer groups, zero points and a bias
        dict(name="int4_decode_m37", op="int4_mm", M=37, N=5120, K=25600, G=64, zeros=True, bias=True),
        # a prompt: the tensor cores decide
        dict(name="int4_prefill_m2048", op="int4_mm", M=2048, N=24576, K=4096, G=128, zeros=False, bias=False),
        # expert products of a decode batch of 8 tokens: about 64 rows over 128 experts
        dict(name="grouped_decode_8", op="grouped_int4_mm", tokens=8, E=EXPERTS, top_k=TOP_K, N=2 * INTER, K=HIDDEN,
             G=128, zeros=False),
        # expert products of a prompt of 1001 tokens, down projection, finest groups
        dict(name="grouped_prefill_1001", op="grouped_int4_mm", tokens=1001, E=EXPERTS, top_k=TOP_K, N=HIDDEN,
             K=INTER, G=32, zeros=True),
        # routing of a small decode batch (ids as torch.topk gives them)
        dict(name="sort_decode_8", op="moe_sort", tokens=8, E=EXPERTS, top_k=TOP_K, bits=64, drop=0.0),
        # routing of a long prompt on one rank of an expert-parallel group: ids of other ranks' experts are -1
        dict(name="sort_prefill_8192", op="moe_sort", tokens=8192, E=EXPERTS, top_k=TOP_K, bits=32, drop=0.25),
        # dispatch of a decode batch with the quantization of its rows
        dict(name="dispatch_fp8_decode_32", op="moe_permute", dir="fwd", fmt="fp8_dynamic", tokens=32, E=EXPERTS,
             top_k=TOP_K, H=HIDDEN, drop=0.0),
        # dispatch's gradient in training
        dict(name="dispatch_bwd_4096", op="moe_permute", dir="bwd", fmt="bf16", tokens=4096, E=EXPERTS, top_k=TOP_K,
             H=HIDDEN, drop=0.0),
        # combination of the experts' rows in a decode step
        dict(name="combine_decode_32", op="moe_unpermute", dir="fwd", tokens=32, E=EXPERTS, top_k=TOP_K, H=HIDDEN,
             drop=0.0),
        # its gradient in training
        dict(name="combine_bwd_4096", op="moe_unpermute", dir="bwd", tokens=4096, E=EXPERTS, top_k=TOP_K, H=HIDDEN,
             drop=0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int4_mm", "int4_mm", "grouped_int4_mm", "moe_sort", "moe_permute", "moe_unpermute"])
    if op == "int4_mm":
        G = rng.choice([32, 64, 128])
        while True:
            M = _log_int(rng, 1, 2048)
            N = 8 * _log_int(rng, 32, 25600 // 8)
            K = G * _log_int(rng, max(1, 256 // G), 25600 // G)
            if 2 * M * N * K <= _MAX_FLOPS:
                break
        return dict(op=op, M=M, N=N, K=K, G=G, zeros=rng.random() < 0.5, bias=rng.random() < 0.3)
    E = rng.choice([8, 60, 64, 128, 160])
    top_k = rng.randint(1, 8)
    if op == "grouped_int4_mm":
        G = rng.choice([32, 64, 128])
        K = G * _log_int(rng, max(1, 256 // G), 2048 // G)
        N = 8 * _log_int(rng, 32, 2048 // 8)
        return dict(op=op, tokens=_log_int(rng, 1, 1001), E=E, top_k=top_k, N=N, K=K, G=G, zeros=rng.random() < 0.5)
    drop = rng.choice([0.0, 0.25])
    if op == "moe_sort":
        return dict(op=op, tokens=_log_int(rng, 1, 8192), E=E, top_k=top_k, bits=rng.choice([32, 64]), drop=drop)
    H = 16 * _log_int(rng, 16, 512)
    tokens = _log_int(rng, 1, 4096)
    tokens = max(1, min(tokens, _MAX_ROWS_BYTES // (H * 2 * (2 * top_k + 1))))
    case = dict(op=op, dir=rng.choice(["fwd", "bwd"]), tokens=tokens, E=E, top_k=top_k, H=H, drop=drop)
    if op == "moe_permute":
        case["fmt"] = rng.choice(["fp8_dynamic", "w8a8_int8", "bf16"]) if case["dir"] == "fwd" else "bf16"
    return case


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(rows, K, g):
    """bf16 N(0, 1) with one channel in a hundred twenty times as large."""
    x = torch.randn((rows, K), generator=g, device="cuda")
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]
    x[:, cols] *= 20.0
    return x.to(torch.bfloat16)


def _int4_weight(rows, K, G, zeros, g):
    """A N(0, 0.02) weight in 4 bits: packed codes [rows, K / 2] (two per
    byte, even k in the low half), bf16 scales and zero points [rows, K / G]."""
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, K // G), dtype=torch.bfloat16, device="cuda")
    zps = torch.empty((rows, K // G), dtype=torch.uint8, device="cuda") if zeros else None
    step = max(1, (1 << 26) // K)
    for r in range(0, rows, step):
        w = torch.randn((min(step, rows - r), K // G, G), generator=g, device="cuda") * 0.02
        lo, hi = w.amin(-1).clamp(max=0.0), w.amax(-1).clamp(min=0.0)
        s = ((hi - lo) / 15.0 if zeros else w.abs().amax(-1) / 7.0).to(torch.bfloat16).float()
        z = (-lo / s).round().clamp(0, 15) if zeros else torch.full_like(s, 8.0)
        q = ((w / s[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).reshape(w.shape[0], K)
        codes[r:r + step] = q[:, 0::2] | (q[:, 1::2] << 4)
        scales[r:r + step] = s.to(torch.bfloat16)
        if zeros:
            zps[r:r + step] = z.to(torch.uint8)
    return codes, scales, zps


def _ids(case, g):
    """Expert ids [tokens, top_k], distinct within a token; -1 with the case's share."""
    T, E, k = case["tokens"], case["E"], case["top_k"]
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices
    if case.get("drop"):
        ids[torch.rand((T, k), generator=g, device="cuda") < case["drop"]] = -1
    return ids


def _routing(ids, E):
    """Offsets [E + 1], order [n] and slots like ids, by counting (int32)."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    hit = flat[:, None] == torch.arange(E, device=ids.device)
    before = hit.to(torch.int32).cumsum(0, dtype=torch.int32)
    ends = before[-1].cumsum(0, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = ends
    kept = (flat >= 0) & (flat < E)
    e = torch.where(kept, flat, torch.zeros_like(flat))
    rank = before.gather(1, e[:, None])[:, 0] - 1
    slots = torch.where(kept, offsets[e] + rank, torch.full_like(rank, -1))
    order = torch.full((n + 1,), -1, dtype=torch.int32, device=ids.device)
    order[torch.where(kept, slots.long(), torch.full_like(flat, n))] = torch.arange(n, dtype=torch.int32,
                                                                                   device=ids.device)
    order[n] = -1
    return offsets, order[:n], slots.reshape(ids.shape)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = dict(case=dict(case))
    if op == "int4_mm":
        st["x"] = _activations(case["M"], case["K"], g)
        st["B"], st["s"], st["z"] = _int4_weight(case["N"], case["K"], case["G"], case["zeros"], g)
        st["bias"] = torch.randn(case["N"], generator=g, device="cuda").to(torch.bfloat16) if case["bias"] else None
        return st
    ids = _ids(case, g)
    if op == "moe_sort":
        st["ids"] = ids.to(torch.int32) if case["bits"] == 32 else ids
        return st
    offsets, order, slots = _routing(ids, case["E"])
    T, k = case["tokens"], case["top_k"]
    if op == "grouped_int4_mm":
        E, N, K, G = case["E"], case["N"], case["K"], case["G"]
        x = _activations(T, K, g)
        st["x"] = x[(order.long() // k)]
        B, s, z = _int4_weight(E * N, K, G, case["zeros"], g)
        st["B"], st["s"] = B.view(E, N, K // 2), s.view(E, N, K // G)
        st["z"] = z.view(E, N, K // G) if z is not None else None
        st["offsets"] = offsets
        st["most"] = int((offsets[1:] - offsets[:-1]).max())   # largest expert: the plain form's padding
        return st
    st["slots"] = slots
    H, P = case["H"], T * k
    if op == "moe_permute" and case["dir"] == "fwd":
        st["x"] = _activations(T, H, g)
        dt = {"bf16": torch.bfloat16, "fp8_dynamic": torch.uint8, "w8a8_int8": torch.int8}[case["fmt"]]
        st["xs"] = torch.zeros((P, H), dtype=dt, device="cuda")     # the program's buffers: rows of dropped
        st["scales"] = torch.zeros(P, device="cuda")                # slots are left as they were
        return st
    if op == "moe_permute":
        st["dxs"] = torch.randn((P, H), generator=g, device="cuda").to(torch.bfloat16)
        return st
    st["y"] = torch.randn((P, H), generator=g, device="cuda").to(torch.bfloat16)
    st["w"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
    if case["dir"] == "bwd":
        st["dout"] = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        st["dy"] = torch.zeros((P, H), dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------- plain forms
def _dequant(B, s, z, dtype):
    """Weights (q - z) * s of packed codes [..., K / 2], as [..., K]."""
    K, groups = B.shape[-1] * 2, s.shape[-1]
    q = torch.stack((B & 15, B >> 4), dim=-1).reshape(*B.shape[:-1], groups, K // groups).to(dtype)
    q = q - (8.0 if z is None else z.to(dtype)[..., None])
    return (q * s.to(dtype)[..., None]).reshape(*B.shape[:-1], K)


def _plain_grouped(st, dtype):
    """Rows of every expert padded to the largest, one batched product."""
    x, off = st["x"].to(dtype), st["offsets"].long()
    T, E = x.shape[0], off.numel() - 1
    row = torch.arange(T, device=x.device)
    e = (row[:, None] >= off[None, 1:]).sum(1)
    pos = e * st["most"] + row - off[e]
    pad = torch.zeros((E * st["most"], x.shape[1]), dtype=dtype, device=x.device)
    pad[pos] = x
    w = _dequant(st["B"], st["s"], st["z"], dtype)
    return torch.bmm(pad.view(E, st["most"], -1), w.transpose(1, 2)).reshape(E * st["most"], -1)[pos]


def _rows(y, slots):
    """y[slots] with zero rows for slots of -1: [T, k, H]."""
    got = y[slots.clamp(min=0).long()]
    return torch.where((slots >= 0)[..., None], got, torch.zeros_like(got))


def _place(buf, slots, rows):
    """A copy of buf with rows [T, k, H] (or [T, k]) written at their slots."""
    P = buf.shape[0]
    out = torch.cat((buf, buf[:1]))
    out[torch.where(slots >= 0, slots, torch.full_like(slots, P)).long().reshape(-1)] = rows.reshape(-1, *rows.shape[2:])
    return out[:P]


def _quantize(x, fmt):
    top = 448.0 if fmt == "fp8_dynamic" else 127.0
    most = x.float().abs().amax(1)
    s = (most / torch.full_like(most, top)).clamp(min=2.0 ** -126)   # by a tensor: the rounded quotient itself
    q = x.float() / s[:, None]
    if fmt == "fp8_dynamic":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), s
    return q.round().clamp(-127, 127).to(torch.int8), s


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "int4_mm":
        c = st["x"].float() @ _dequant(st["B"], st["s"], st["z"], torch.float32).t()
        return (c if st["bias"] is None else c + st["bias"].float()).to(torch.bfloat16)
    if op == "grouped_int4_mm":
        return _plain_grouped(st, torch.float32).to(torch.bfloat16)
    if op == "moe_sort":
        return _routing(st["ids"], case["E"])
    slots = st["slots"]
    k = case["top_k"]
    if op == "moe_permute" and case["dir"] == "fwd":
        if case["fmt"] == "bf16":
            return _place(st["xs"], slots, st["x"][:, None].expand(-1, k, -1))
        q, s = _quantize(st["x"], case["fmt"])
        return _place(st["xs"], slots, q[:, None].expand(-1, k, -1)), _place(st["scales"], slots, s[:, None].expand(-1, k))
    if op == "moe_permute":
        return _rows(st["dxs"], slots).float().sum(1).to(torch.bfloat16)
    if case["dir"] == "fwd":
        return (_rows(st["y"], slots).float() * st["w"][..., None]).sum(1).to(torch.bfloat16)
    d = st["dout"].float()[:, None]
    dw = (_rows(st["y"], slots).float() * d).sum(2)
    return _place(st["dy"], slots, (d * st["w"][..., None]).to(torch.bfloat16)), dw


# --------------------------------------------------------- library's calls
def _own(st):
    from quantized_linear_gemm_b200 import lq
    case = st["case"]
    op = case["op"]
    if op == "int4_mm":
        return lq.int4_mm(st["x"], st["B"], st["s"], b_zeros=st["z"], bias=st["bias"])
    if op == "grouped_int4_mm":
        return lq.grouped_int4_mm(st["x"], st["B"], st["s"], st["offsets"], b_zeros=st["z"])
    if op == "moe_sort":
        return lq.moe_sort(st["ids"], case["E"])
    slots = st["slots"]
    if op == "moe_permute" and case["dir"] == "fwd":
        if case["fmt"] == "bf16":
            return lq.moe_permute(st["x"], slots, xs=st["xs"])
        return lq.moe_permute_quant(case["fmt"], st["x"], slots, q=st["xs"], scales=st["scales"])
    if op == "moe_permute":
        return lq.moe_permute_backward(st["dxs"], slots)
    if case["dir"] == "fwd":
        return lq.moe_unpermute(st["y"], slots, st["w"])
    return lq.moe_unpermute_backward(st["dout"], st["y"], slots, st["w"], dy=st["dy"])


def _values(case, out):
    """e4m3 codes as the values that they stand for (a view, no work)."""
    if case.get("fmt") == "fp8_dynamic":
        return out[0].view(torch.float8_e4m3fn), out[1]
    return out


def run(state):
    return _values(state["case"], _own(state) if own else _plain(state))


def work(case):
    op = case["op"]
    if op == "int4_mm":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        b = N * K // 2 + N * (K // G) * (3 if case["zeros"] else 2) + 2 * M * K + 2 * M * N + (2 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * N * K}
    T, E, k = case["tokens"], case["E"], case["top_k"]
    P = T * k
    if op == "grouped_int4_mm":
        N, K, G = case["N"], case["K"], case["G"]
        used = E * (1.0 - (1.0 - k / E) ** T)      # experts with rows, on average
        per = N * K // 2 + N * (K // G) * (3 if case["zeros"] else 2)
        return {"bytes": int(used * per) + 2 * P * K + 2 * P * N + 4 * (E + 1), "flops": 2 * P * N * K}
    if op == "moe_sort":
        return {"bytes": P * (case["bits"] // 8 + 8) + 4 * (E + 1), "flops": 0}
    H = case["H"]
    kept = int(P * (1.0 - case["drop"]))
    if op == "moe_permute" and case["dir"] == "fwd":
        out = 2 * H if case["fmt"] == "bf16" else H + 4
        return {"bytes": 2 * T * H + kept * out + 4 * P, "flops": 0 if case["fmt"] == "bf16" else 3 * T * H}
    if op == "moe_permute":
        return {"bytes": 2 * T * H + 2 * kept * H + 4 * P, "flops": kept * H}
    if case["dir"] == "fwd":
        return {"bytes": 2 * T * H + 2 * kept * H + 8 * P, "flops": 2 * kept * H}
    return {"bytes": 2 * T * H + 4 * kept * H + 12 * P, "flops": 3 * kept * H}


# ------------------------------------------------------------ in 64 bits
def _weights64(B, s, z):
    """The weights of packed codes in fp64, a nibble plane at a time."""
    rows, groups = B.reshape(-1, B.shape[-1]), s.reshape(-1, s.shape[-1])
    out = torch.empty((rows.shape[0], 2 * rows.shape[1]), dtype=torch.float64, device=B.device)
    out[:, 0::2] = (rows % 16).double()
    out[:, 1::2] = torch.div(rows, 16, rounding_mode="floor").double()
    G = out.shape[1] // groups.shape[1]
    out -= z.reshape(groups.shape).double().repeat_interleave(G, dim=1) if z is not None else 8.0
    out *= groups.double().repeat_interleave(G, dim=1)
    return out


def _e4m3_64(v):
    """fp64 values on the e4m3 grid: half a step to even, at most 448."""
    a = v.abs()
    e = torch.floor(torch.log2(torch.clamp(a, min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > a, torch.clamp(e - 1, min=-6.0), e)
    e = torch.where(torch.exp2(e + 1) <= a, e + 1, e)
    step = torch.exp2(e - 3)
    return torch.copysign(torch.clamp(torch.round(a / step) * step, max=448.0), v)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "int4_mm":
        c = st["x"].double() @ _weights64(st["B"], st["s"], st["z"]).t()
        return c if st["bias"] is None else c + st["bias"].double()
    if op == "grouped_int4_mm":
        off = st["offsets"].tolist()
        w = _weights64(st["B"], st["s"], st["z"]).view(case["E"], case["N"], case["K"])
        return torch.cat([st["x"][a:b].double() @ w[e].t() for e, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    if op == "moe_sort":
        ids = st["ids"].reshape(-1)
        key = torch.where((ids < 0) | (ids >= case["E"]), torch.full_like(ids, case["E"]), ids)
        order = torch.argsort(key, stable=True)
        n = int((key < case["E"]).sum())
        offsets = torch.searchsorted(key[order], torch.arange(case["E"] + 1, device="cuda", dtype=key.dtype))
        slots = torch.full_like(order, -1)
        slots[order[:n]] = torch.arange(n, device="cuda")
        order[n:] = -1
        return offsets.int(), order.int(), slots.int().reshape(st["ids"].shape)
    slots = st["slots"].reshape(-1).long()
    T, k, H = case["tokens"], case["top_k"], case["H"]
    kept = torch.nonzero(slots >= 0)[:, 0]
    at = slots[kept]
    if op == "moe_permute" and case["dir"] == "fwd":
        src = st["x"].double()[kept // k]
        xs = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
        if case["fmt"] == "bf16":
            xs[at] = src
            return xs
        top = 448.0 if case["fmt"] == "fp8_dynamic" else 127.0
        s = (src.abs().amax(1) / top).float().clamp(min=2.0 ** -126)
        v = (src / s.double()[:, None]).float().double()      # the quotient is rounded to 32 bits by definition
        scales = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        scales[at] = s.double()
        if case["fmt"] == "fp8_dynamic":
            xs[at] = _e4m3_64(v)
            return xs, scales
        codes = torch.zeros((T * k, H), dtype=torch.int8, device="cuda")
        codes[at] = torch.round(v).clamp(-127, 127).to(torch.int8)
        return codes, scales
    if op == "moe_permute":
        dx = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        return dx.index_add_(0, kept // k, st["dxs"].double()[at])
    w = st["w"].double().reshape(-1)
    if case["dir"] == "fwd":
        out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
        return out.index_add_(0, kept // k, st["y"].double()[at] * w[kept][:, None])
    d = st["dout"].double()[kept // k]
    dy = torch.zeros((T * k, H), dtype=torch.float64, device="cuda")
    dy[at] = d * w[kept][:, None]
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    dw[kept] = (d * st["y"].double()[at]).sum(1)
    return dy, dw.reshape(T, k)
