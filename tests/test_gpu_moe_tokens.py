"""GPU parity of the mixture-of-experts token movement against the CPU oracle:
sort, dispatch (bf16 and quantized), combination and the gradients, and a
whole expert layer from router ids to combined rows.

Tolerances, derived (r exact in fp64, S the sum of the magnitudes of its
terms): a sum of n fp32 fused multiply-adds is off by at most n 2^-23 S, a
rounding to bf16 by half a step, 2^-8 of the value.  dy is one fp32 product
(2^-24) rounded to bf16."""

import numpy as np
import pytest
import torch

from oracle import lq_oracle as O
from oracle import moe_oracle as MO
from oracle import moe_tokens_oracle as T
from oracle import producer_oracle as P
from quantized_linear_gemm_b200 import inputs, lq

from _lqtest import bf16_to_f64

pytestmark = pytest.mark.gpu


def routing(tokens, k, E, seed, drop=0.0, crowd=False):
    g = np.random.default_rng(seed)
    ids = np.stack([g.choice(E, size=k, replace=False) if k <= E else g.integers(0, E, k) for _ in range(tokens)]) \
        if tokens else np.zeros((0, k), dtype=np.int64)
    if crowd:
        ids[:, 0] = E - 1
    ids = ids.astype(np.int64)
    ids[g.random(ids.shape) < drop] = -1
    return ids


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,E", [(0, 2, 4), (1, 1, 1), (1, 8, 128), (5, 3, 7), (33, 4, 60), (128, 8, 128),
                                        (1025, 1, 8), (1000, 6, 257), (3001, 8, 1024), (9000, 8, 64)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_sort(cuda_device, dtype, tokens, k, E, drop):
    ids = routing(tokens, k, E, seed=tokens + E, drop=drop)
    off, order, slots = lq.moe_sort(cuda(ids, dtype), E)
    torch.cuda.synchronize()
    ro, rr, rs = T.moe_sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro)
    assert np.array_equal(slots.cpu().numpy(), rs)
    assert np.array_equal(order.cpu().numpy(), rr)


@pytest.mark.parametrize("kind", ["one", "none", "outside"])
def test_sort_extremes(cuda_device, kind):
    """Every id the same, none routed, and ids far outside the range (64-bit ones whose low half is a valid id)."""
    E, n = 16, 5000
    ids = {"one": np.full(n, 5), "none": np.full(n, -1),
           "outside": np.tile(np.array([3, 16, -7, 2 ** 32 + 3, -2 ** 40, 15, 2 ** 62, 0]), n // 8)}[kind]
    ids = ids.astype(np.int64).reshape(-1, 4)
    off, order, slots = lq.moe_sort(cuda(ids), E)
    torch.cuda.synchronize()
    ro, rr, rs = T.moe_sort(ids, E)
    assert np.array_equal(off.cpu().numpy(), ro) and np.array_equal(order.cpu().numpy(), rr)
    assert np.array_equal(slots.cpu().numpy(), rs)


SHAPES = [(1, 1, 16), (1, 8, 2048), (3, 2, 272), (37, 8, 2048), (20, 9, 1040), (5, 17, 4112), (4, 3, 17424)]


def case(tokens, k, H, seed=0, drop=0.2):
    E = 19
    ids = routing(tokens, k, E, seed=seed + tokens, drop=drop)
    off, order, slots = T.moe_sort(ids, E)
    return off, order, slots


@pytest.mark.parametrize("tokens,k,H", SHAPES)
def test_permute(cuda_device, tokens, k, H):
    _, _, slots = case(tokens, k, H)
    x = inputs.activations(tokens, H, seed=H)
    for rows in (tokens * k, max(1, tokens * k // 2)):          # a buffer shorter than the slots: the rest is skipped
        base = torch.full((rows + 1, H), 3.0, dtype=torch.bfloat16)
        buf = base.cuda()
        lq.moe_permute(x.cuda(), cuda(slots), xs=buf[:rows])
        torch.cuda.synchronize()
        ref = T.permute(x.float().numpy(), slots, base[:rows].float().numpy())
        assert np.array_equal(buf[:rows].float().cpu().numpy(), ref)
        assert torch.all(buf[rows:] == 3.0)


@pytest.mark.parametrize("fmt", ["fp8_dynamic", "w8a8_int8"])
@pytest.mark.parametrize("tokens,k,H", SHAPES)
def test_permute_quant(cuda_device, fmt, tokens, k, H):
    """Bit for bit the oracle's codes and scales at every slot; other rows as they were."""
    _, _, slots = case(tokens, k, H)
    x = inputs.activations(tokens, H, seed=H + 1)
    x[0] = 0
    codes, scales = O.quant_per_token(x.float().numpy(), fmt)
    n = tokens * k
    q = torch.full((n, H), 77, dtype=torch.int8 if fmt == "w8a8_int8" else torch.uint8, device="cuda")
    s = torch.full((n,), 5.0, device="cuda")
    lq.moe_permute_quant(fmt, x.cuda(), cuda(slots), q=q, scales=s)
    torch.cuda.synchronize()
    assert np.array_equal(q.cpu().numpy(), T.permute(codes, slots, np.full((n, H), 77, codes.dtype)))
    assert np.array_equal(s.cpu().numpy(), T.permute(scales, slots, np.full(n, 5.0, np.float32)))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("tokens,k,H", SHAPES)
def test_unpermute(cuda_device, tokens, k, H, weighted):
    _, _, slots = case(tokens, k, H)
    n = tokens * k
    g = torch.Generator().manual_seed(H)
    y = torch.randn((n, H), generator=g).bfloat16()
    named = np.zeros(n, dtype=bool)
    named[slots[slots >= 0]] = True
    y[torch.from_numpy(~named)] = float("nan")                   # rows that no slot names are never read
    w = torch.randn((tokens, k), generator=g)
    w[torch.from_numpy(slots < 0)] = float("inf")                # nor do skipped weights count
    if weighted:
        out = lq.moe_unpermute(y.cuda(), cuda(slots), w.cuda())
    else:
        out = lq.moe_permute_backward(y.cuda(), cuda(slots))
    torch.cuda.synchronize()
    yr = y.float().numpy()
    yr[~named] = 0
    wr = np.where(slots < 0, 0, w.numpy())
    r, mag = T.unpermute(yr, slots, wr if weighted else None)
    e = k * 2.0 ** -23 * mag
    assert np.all(np.abs(bf16_to_f64(out) - r) <= e + 2.0 ** -8 * (np.abs(r) + e))


@pytest.mark.parametrize("tokens,k,H", SHAPES)
def test_unpermute_backward(cuda_device, tokens, k, H):
    _, _, slots = case(tokens, k, H)
    n = tokens * k
    g = torch.Generator().manual_seed(H + 5)
    y, dout = torch.randn((n, H), generator=g).bfloat16(), torch.randn((tokens, H), generator=g).bfloat16()
    w = torch.randn((tokens, k), generator=g)
    dy = torch.full((n, H), 3.0, dtype=torch.bfloat16, device="cuda")
    dy, dw = lq.moe_unpermute_backward(dout.cuda(), y.cuda(), cuda(slots), w.cuda(), dy=dy)
    torch.cuda.synchronize()
    rdy, rdw, mag = T.unpermute_backward(dout.float().numpy(), y.float().numpy(), slots, w.numpy(),
                                         np.full((n, H), 3.0))
    assert np.all(np.abs(bf16_to_f64(dy) - rdy) <= np.abs(rdy) * (2.0 ** -8 + 2.0 ** -23))
    assert np.all(np.abs(dw.cpu().numpy() - rdw) <= H * 2.0 ** -23 * mag)


def test_gradients_agree_with_differences(cuda_device):
    """The kernels' own outputs: out is linear in y and in the weights, so a
    difference of two outputs along one row or one weight gives its gradient.
    Inputs are small whole numbers, for which every product, sum and rounding
    here is exact."""
    tokens, k, H, E = 6, 3, 64, 5
    ids = routing(tokens, k, E, seed=1, drop=0.2)
    off, order, slots = lq.moe_sort(cuda(ids), E)
    g = torch.Generator().manual_seed(2)
    small = lambda *shape: torch.randint(-2, 3, shape, generator=g).float()   # noqa: E731
    y, dout, w = small(tokens * k, H).bfloat16().cuda(), small(tokens, H).bfloat16().cuda(), small(tokens, k).cuda()
    dy, dw = lq.moe_unpermute_backward(dout, y, slots, w, dy=torch.zeros_like(y))
    base = lq.moe_unpermute(y, slots, w).double()
    for p in range(tokens * k):
        step = torch.zeros_like(y)
        step[p] = small(H).bfloat16().cuda()
        diff = ((lq.moe_unpermute(y + step, slots, w).double() - base) * dout.double()).sum()
        assert float(diff) == float((dy.double() * step.double()).sum())
    for t in range(tokens):
        for j in range(k):
            step = torch.zeros_like(w)
            step[t, j] = 1.0
            diff = ((lq.moe_unpermute(y, slots, w + step).double() - base) * dout.double()).sum()
            assert float(diff) == float(dw[t, j])
    dxs = small(tokens * k, H).bfloat16().cuda()
    dx = lq.moe_permute_backward(dxs, slots)
    x = small(tokens, H).bfloat16().cuda()
    xs = lq.moe_permute(x, slots, xs=torch.zeros_like(dxs)).double()
    for t in range(tokens):
        step = torch.zeros_like(x)
        step[t] = small(H).bfloat16().cuda()
        diff = ((lq.moe_permute(x + step, slots, xs=torch.zeros_like(dxs)).double() - xs) * dxs.double()).sum()
        assert float(diff) == float((dx.double() * step.double()).sum())


def test_repeatable_and_graph_replay(cuda_device):
    tokens, k, E, H = 300, 8, 64, 512
    ids = cuda(routing(tokens, k, E, seed=3, drop=0.1))
    x = inputs.activations(tokens, H, seed=1).cuda()
    w = torch.rand((tokens, k), device="cuda")
    off, order, slots = lq.moe_sort(ids, E)
    xs = lq.moe_permute(x, slots, xs=torch.zeros((tokens * k, H), dtype=torch.bfloat16, device="cuda"))
    out = lq.moe_unpermute(xs, slots, w)
    dy, dw = lq.moe_unpermute_backward(x, xs, slots, w, dy=torch.zeros_like(xs))
    st = torch.cuda.Stream()
    o2, r2, s2 = torch.empty_like(off), torch.empty_like(order), torch.empty_like(slots)
    xs2, out2, dy2, dw2 = torch.zeros_like(xs), torch.empty_like(out), torch.zeros_like(dy), torch.empty_like(dw)

    def chain():
        lq.moe_sort(ids, E, o2, r2, s2)
        lq.moe_permute(x, s2, xs=xs2)
        lq.moe_unpermute(xs2, s2, w, out=out2)
        lq.moe_unpermute_backward(x, xs2, s2, w, dy=dy2, dweights=dw2)

    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        chain()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            chain()
    for t in (o2, r2, s2, xs2, out2, dy2, dw2):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in ((off, o2), (order, r2), (slots, s2), (xs, xs2), (out, out2), (dy, dy2), (dw, dw2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("drop", [0.0, 0.25])
def test_fp8_expert_layer(cuda_device, drop):
    """Router ids to combined rows with FP8 experts, as a serving step runs it,
    against the oracles chained in the same order (codes bit for bit)."""
    tokens, k, E, H, I = 9, 4, 12, 256, 128
    ids = routing(tokens, k, E, seed=11, drop=drop)
    x = inputs.activations(tokens, H, seed=12)
    w = torch.softmax(torch.randn((tokens, k), generator=torch.Generator().manual_seed(13)), 1)
    gu = inputs.weights(E * 2 * I, H, seed=14).float().numpy().reshape(E, 2 * I, H)
    dn = inputs.weights(E * H, I, seed=15).float().numpy().reshape(E, H, I)
    fmt = "fp8_dynamic"
    qgu, sgu = zip(*(O.quant_per_channel(m, fmt) for m in gu))
    qdn, sdn = zip(*(O.quant_per_channel(m, fmt) for m in dn))
    qgu, sgu, qdn, sdn = (np.stack(a) for a in (qgu, sgu, qdn, sdn))

    off, order, slots = lq.moe_sort(cuda(ids), E)
    n = tokens * k
    q, s = lq.moe_permute_quant(fmt, x.cuda(), slots, q=torch.zeros((n, H), dtype=torch.uint8, device="cuda"),
                                scales=torch.ones(n, device="cuda"))
    h = lq.grouped_scaled_mm(fmt, q, s, cuda(qgu), cuda(sgu.astype(np.float32)), off,
                             C=torch.zeros((n, 2 * I), dtype=torch.bfloat16, device="cuda"))
    qh, sh = lq.silu_and_mul_dynamic_per_token_quant(fmt, h)
    y = lq.grouped_scaled_mm(fmt, qh, sh, cuda(qdn), cuda(sdn.astype(np.float32)), off,
                             C=torch.full((n, H), float("nan"), dtype=torch.bfloat16, device="cuda"))
    out = lq.moe_unpermute(y, slots, w.cuda())
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0

    ro, _, rs = T.moe_sort(ids, E)
    codes, scales = O.quant_per_token(x.float().numpy(), fmt)
    kept = int(ro[-1])
    rq = T.permute(codes, rs, np.zeros((n, H), codes.dtype))
    rsc = T.permute(scales, rs, np.ones(n, np.float32))
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rsc)
    rh = MO.grouped_scaled_mm_ref(fmt, rq[:kept], rsc[:kept], qgu, sgu, ro)
    ok, worst = O.within_tolerance(bf16_to_f64(h[:kept]), rh)
    assert ok, worst
    pq, ps = P.silu_and_mul_dynamic_per_token_quant(bf16_to_f64(h[:kept]), fmt)[:2]   # from the kernel's own h
    assert np.array_equal(qh[:kept].cpu().numpy(), pq) and np.array_equal(sh[:kept].cpu().numpy(), ps)
    ry = MO.grouped_scaled_mm_ref(fmt, pq, ps, qdn, sdn, ro)
    ok, worst = O.within_tolerance(bf16_to_f64(y[:kept]), ry)
    assert ok, worst
    yk = np.zeros((n, H))
    yk[:kept] = bf16_to_f64(y[:kept])
    r, mag = T.unpermute(yk, rs, w.numpy())
    e = k * 2.0 ** -23 * mag
    assert np.all(np.abs(bf16_to_f64(out) - r) <= e + 2.0 ** -8 * (np.abs(r) + e))


def test_int4_expert_layer(cuda_device):
    """The same movement around 4-bit experts: sort, dispatch in bf16, grouped
    4-bit product, weighted combination; each step against its oracle."""
    from oracle import int4_oracle as I4
    tokens, k, E, H, N, group = 21, 2, 6, 384, 264, 64
    ids = routing(tokens, k, E, seed=21, drop=0.2)
    x = inputs.activations(tokens, H, seed=22)
    wt = inputs.weights(E * N, H, seed=23)
    w = torch.rand((tokens, k), generator=torch.Generator().manual_seed(24))
    B, s, z = lq.quant_weight_int4(wt.cuda(), group, zero_points=True)
    off, order, slots = lq.moe_sort(cuda(ids), E)
    xs = lq.moe_permute(x.cuda(), slots)
    y = lq.grouped_int4_mm(xs, B.view(E, N, -1), s.view(E, N, -1), off, b_zeros=z.view(E, N, -1))
    out = lq.moe_unpermute(y, slots, w.cuda())
    torch.cuda.synchronize()
    assert lq.device_status(0) == 0
    wd = I4.dequant(B.cpu().numpy(), s.float().cpu().numpy(), z.cpu().numpy()).reshape(E, N, H)
    ro, _, rs = T.moe_sort(ids, E)
    r = np.zeros((tokens, N))
    mag = np.zeros((tokens, N))
    for t in range(tokens):
        for j in range(k):
            if ids[t, j] >= 0:
                xt = x[t].float().numpy().astype(np.float64)
                r[t] += float(w[t, j]) * (wd[ids[t, j]] @ xt)
                mag[t] += abs(float(w[t, j])) * (np.abs(wd[ids[t, j]]) @ np.abs(xt))
    # y is off by at most H 2^-23 S and half a bf16 step; the combination adds its own k terms and one rounding
    e = (H * 2.0 ** -23 + 2.0 ** -8 * (1 + H * 2.0 ** -23) + k * 2.0 ** -22) * mag
    assert np.all(np.abs(bf16_to_f64(out) - r) <= e + 2.0 ** -8 * (np.abs(r) + e))


def test_rows_past_2_31_elements(cuda_device):
    """Slots whose rows lie past 2^31 elements: dispatch, combination and the gradients against torch indexing."""
    tokens, k, H = 140000, 8, 2048
    n = tokens * k
    assert n * H > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.rand((tokens, 16), generator=g, device="cuda").topk(k, 1).indices
    off, order, slots = lq.moe_sort(ids, 16)
    assert int(off[-1]) == n
    flat = ids.reshape(-1)
    assert torch.equal(order.long(), torch.argsort(flat, stable=True))
    x = torch.randn((tokens, H), generator=g, device="cuda").bfloat16()
    xs = lq.moe_permute(x, slots)
    pick = torch.randint(0, n, (4000,), generator=g, device="cuda")
    pick[0], pick[1] = n - 1, 0
    assert torch.equal(xs[pick], x[order[pick].long() // k])
    w = torch.full((tokens, k), 0.125, device="cuda")
    assert torch.equal(lq.moe_unpermute(xs, slots, w), x)        # eight equal rows of weight 1/8: exact
    dy, dw = lq.moe_unpermute_backward(x, xs, slots, w)
    assert torch.equal(dy[pick], (x[order[pick].long() // k].float() * 0.125).bfloat16())
    t = torch.randint(0, tokens, (50,), generator=g, device="cuda")
    ref = (x[t].double() ** 2).sum(1)[:, None].expand(-1, k)
    assert torch.all((dw[t].double() - ref).abs() <= H * 2.0 ** -23 * ref)


def test_tokens_without_slots(cuda_device):
    """k = 0: nothing to sum; no tokens: nothing to do."""
    y = torch.randn((4, 64), device="cuda").bfloat16()
    out = lq.moe_unpermute(y, torch.empty((3, 0), dtype=torch.int32, device="cuda"))
    assert out.shape == (3, 64) and torch.all(out == 0)
    assert lq.moe_permute(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
                          torch.empty((0, 2), dtype=torch.int32, device="cuda")).shape == (0, 64)


def test_slots_outside_the_rows_are_skipped(cuda_device):
    """Slots past the last row or negative: neither read nor written (a short buffer, a foreign table)."""
    tokens, k, H, P = 6, 3, 128, 10
    g = np.random.default_rng(3)
    slots = g.permutation(np.arange(-4, 14))[: tokens * k].reshape(tokens, k).astype(np.int32)
    slots[0] = [2 ** 31 - 1, -2 ** 31, 10]
    x = inputs.activations(tokens, H, seed=1)
    y = inputs.activations(P, H, seed=2)
    w = torch.rand((tokens, k), generator=torch.Generator().manual_seed(3))
    base = torch.full((P + 2, H), 3.0, dtype=torch.bfloat16, device="cuda")
    buf = base.clone()
    lq.moe_permute(x.cuda(), cuda(slots), xs=buf[:P])
    assert np.array_equal(buf[:P].float().cpu().numpy(), T.permute(x.float().numpy(), slots, np.full((P, H), 3.0)))
    assert torch.all(buf[P:] == 3.0)
    out = lq.moe_unpermute(y.cuda(), cuda(slots), w.cuda())
    r, mag = T.unpermute(y.float().numpy(), slots, w.numpy())
    e = k * 2.0 ** -23 * mag
    assert np.all(np.abs(bf16_to_f64(out) - r) <= e + 2.0 ** -8 * (np.abs(r) + e))
    buf = base.clone()
    dy, dw = lq.moe_unpermute_backward(x.cuda(), y.cuda(), cuda(slots), w.cuda(), dy=buf[:P])
    rdy, rdw, mag = T.unpermute_backward(x.float().numpy(), y.float().numpy(), slots, w.numpy(), np.full((P, H), 3.0))
    assert np.all(np.abs(bf16_to_f64(dy) - rdy) <= np.abs(rdy) * (2.0 ** -8 + 2.0 ** -23))
    assert np.all(np.abs(dw.cpu().numpy() - rdw) <= H * 2.0 ** -23 * mag) and torch.all(buf[P:] == 3.0)


@pytest.mark.parametrize("op", ["sort", "permute", "unpermute", "backward"])
def test_inputs_written_just_before(cuda_device, op):
    """Each call reads what the kernel before it on the stream wrote (the launches overlap in part)."""
    tokens, k, E, H = 64, 4, 8, 512
    ids = [cuda(routing(tokens, k, E, seed=s)) for s in (1, 2)]
    slots = [lq.moe_sort(i, E)[2] for i in ids]
    x = [inputs.activations(tokens, H, seed=s).cuda() for s in (1, 2)]
    y = [inputs.activations(tokens * k, H, seed=s).cuda() for s in (3, 4)]
    w = torch.rand((tokens, k), device="cuda")
    run = {"sort": lambda i, sl, x, y: lq.moe_sort(i, E), "permute": lambda i, sl, x, y: (lq.moe_permute(x, sl),),
           "unpermute": lambda i, sl, x, y: (lq.moe_unpermute(y, sl, w),),
           "backward": lambda i, sl, x, y: lq.moe_unpermute_backward(x, y, sl, w)}[op]
    torch.cuda.synchronize()
    want = []
    for i in (0, 1):
        want.append([t.clone() for t in run(ids[i], slots[i], x[i], y[i])])
        torch.cuda.synchronize()
    bufs = [torch.empty_like(t[0]) for t in (ids, slots, x, y)]
    for n in range(20):
        i = n & 1
        for b, t in zip(bufs, (ids, slots, x, y)):
            b.copy_(t[i])
        got = run(*bufs)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
