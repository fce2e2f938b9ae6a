"""GPU tests of the experts' rows and of the Sparse-MoE FFN on 4-bit experts: the order bit for bit,
sums within the bound of a float32 sum of that many terms and half a step of the output's type,
gradients against the formula's and against differences."""
from __future__ import annotations

import pytest
import torch

from rankmixer_feature_interaction_gb300 import _lib
from rankmixer_feature_interaction_gb300.api import (Fp4MoE, expert_combine, expert_combine_backward, expert_gather,
                                                     expert_gather_backward, expert_sort, fp4_dequantize,
                                                     fp4_expert_gather, fp4_expert_matmul, fp4_quantize, fp8_sync_status)
from tests import fp4_reference as ref
from tests.test_gpu_fp4 import DEV, DTYPES, gen, layer, ok, rows, within

pytestmark = pytest.mark.gpu
HALF = {"bf16": ref.HALF_BF16, "f32": ref.UNIT_F32}


def gates(B, T, E, share, seed):
    g = gen(seed)
    G = torch.rand((B, T, E), generator=g) - (1 - share) * (0.5 + torch.rand((1, T, E), generator=g))
    return torch.relu(G)


SORTS = [(1, 1, 1), (1, 3, 5), (8, 32, 8), (64, 32, 8), (65, 32, 8), (64, 3, 90), (63, 1, 1), (130, 1, 1), (129, 5, 7),
         (500, 2, 33), (1000, 3, 4), (4100, 1, 9), (257, 16, 40), (2, 700, 12), (3000, 4, 2), (4, 400, 10), (70000, 1, 3),
         (20001, 2, 12), (2049, 1, 64)]


@pytest.mark.parametrize("B,T,E", SORTS)
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_sort(B, T, E, share):
    G = gates(B, T, E, share, 1) if share < 1 else torch.ones((B, T, E))
    if share == 0:
        G = torch.zeros((B, T, E))
    r = expert_sort(G.to(DEV))
    offsets, source, slot = ref.sorted_rows(G)
    n = len(source)
    assert r.count() == n and torch.equal(r.offsets.cpu(), offsets) and torch.equal(r.slot.cpu(), slot)
    assert torch.equal(r.source[:n].cpu(), source)
    ok()


def test_sort_of_special_gates():
    G = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0, 0.0, 2.0 ** -149, -1.0, 1.0]).repeat(70, 1, 1)
    for B in (3, 70):
        r = expert_sort(G[:B].to(DEV))
        assert r.offsets.cpu().diff().tolist() == [0, B, 0, 0, 0, B, 0, B]


def test_sort_leaves_the_rest_of_source_alone():
    G = gates(90, 4, 3, 0.4, 2).to(DEV)
    r = expert_sort(G)
    n = r.count()
    r.source.fill_(-7)
    work = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    _lib.rm_expert_sort(G.data_ptr(), r.c, work.data_ptr(), 1 << 16, torch.cuda.current_stream().cuda_stream)
    assert (r.source[n:] == -7).all() and (r.source[:n] >= 0).all() and n < r.source.numel()


ROWS = [(1, 1, 1, 1), (3, 2, 5, 4), (8, 4, 768, 8), (70, 3, 1003, 6), (5, 2, 40, 40), (130, 5, 264, 3), (9, 1, 2056, 33),
        (2, 1, 4099, 2)]
# rows that a part of a warp takes, with more and fewer experts than its lanes
ROWS += [(131, 3, 100, 19), (37, 5, 64, 17), (1201, 7, 24, 11), (333, 3, 320, 9), (1, 3, 192, 8), (59, 1, 65, 5), (23, 3, 128, 65)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,E", ROWS)
def test_rows_there_and_back(B, T, D, E, dtype):
    dt, g = DTYPES[dtype], gen(4)
    G = gates(B, T, E, 0.5, 3)
    r = expert_sort(G.to(DEV))
    _, source, slot = ref.sorted_rows(G)
    n, at = len(source), source.long()
    X = torch.randn((B, T, D), generator=g).to(dt)
    Y, dXs = (torch.randn((n, D), generator=g).to(dt) for _ in range(2))
    dV = torch.randn((B, T, D), generator=g).to(dt)

    Xs = expert_gather(X.to(DEV), r)
    assert Xs.shape[0] == B * T * E and torch.equal(Xs[:n].cpu(), X.view(-1, D)[at])
    assert torch.equal(expert_gather(X.to(DEV), r, n), Xs[:n])

    def spread(Z):                                   # [B, T, E, D], zero where closed
        full = torch.zeros((B, T, E, D), dtype=torch.float64)
        full[slot >= 0] = Z.double()[slot[slot >= 0].long()]
        return full
    Gd = G.double().unsqueeze(-1)
    V = expert_combine(Y.to(DEV), r, G.to(DEV)).cpu()
    want, bound = (Gd * spread(Y)).sum(2), ref.sum_bound(E, (Gd * spread(Y)).abs().sum(2))
    within(V, want, bound + (want.abs() + bound) * HALF[dtype], "combine")
    assert (V[(slot < 0).all(-1)] == 0).all()
    for out in ("f32", "bf16"):
        within(expert_combine(Y.to(DEV), r, G.to(DEV), out_dtype=out).cpu(), want, bound + (want.abs() + bound) * HALF[out], out)
    dX = expert_gather_backward(dXs.to(DEV), r).cpu()
    want, bound = spread(dXs).sum(2), ref.sum_bound(E, spread(dXs).abs().sum(2))
    within(dX, want, bound + (want.abs() + bound) * HALF[dtype], "gather's gradient")
    dY, dG = (v.cpu() for v in expert_combine_backward(dV.to(DEV), Y.to(DEV), r, G.to(DEV)))
    want = G.double().transpose(0, 1).transpose(1, 2)[(slot >= 0).permute(1, 2, 0)].unsqueeze(-1) * dV.double().view(-1, D)[at]
    within(dY, want, want.abs() * (HALF[dtype] + ref.UNIT_F32) + 1e-300, "dY")
    prod = spread(Y) * dV.double().unsqueeze(2)
    within(dG, prod.sum(-1), ref.sum_bound(D, prod.abs().sum(-1)), "dG")
    assert (dG[slot < 0] == 0).all()
    # the gradient against differences: V is linear in Y and in the open gates
    loss = lambda y, gg: (spread(y) * gg.double().unsqueeze(-1)).sum(2).mul(dV.double()).sum()      # noqa: E731
    hY, hG = torch.randn((n, D), generator=g, dtype=torch.float64), torch.randn((B, T, E), generator=g) * (slot >= 0)
    for h in ((hY, 0 * hG), (0 * hY, hG)):
        step = (loss(Y.double() + h[0], G + h[1]) - loss(Y.double() - h[0], G - h[1])) / 2
        got = (dY.double() * h[0]).sum() + (dG.double() * h[1].double()).sum()
        tol = (dY.double() * h[0]).abs().sum() * 2 * HALF[dtype] + \
            (ref.sum_bound(D, prod.abs().sum(-1)) * h[1].double().abs()).sum() + 1e-5 * (G + h[1].abs()).max() * prod.abs().sum()
        assert (step - got).abs() <= tol
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 37])
def test_room_for_fewer_rows(D, dtype):
    """Slots without room count as closed, and nothing is written behind the rows."""
    B, T, E, dt = 40, 3, 4, DTYPES[dtype]
    G = gates(B, T, E, 0.6, 5).to(DEV)
    r = expert_sort(G)
    n = r.count()
    X, dV = rows((B, T, D), 6).to(dt).to(DEV), rows((B, T, D), 7).to(dt).to(DEV)
    Y = rows((n, D), 8).to(dt).to(DEV)
    for room in (0, 1, n // 2, n, n + 9):
        m = min(room, n)
        closed = torch.where((r.slot >= 0) & (r.slot < room), G, torch.zeros_like(G))
        stream = torch.cuda.current_stream().cuda_stream
        buf = torch.full((room + 3, D), 5.0, dtype=dt, device=DEV)
        _lib.rm_expert_gather(X.data_ptr(), int(dt is torch.bfloat16), r.c, buf.data_ptr(), room, D, stream)
        assert torch.equal(buf[:m], expert_gather(X, r)[:m]) and (buf[m:] == 5).all()
        V = expert_combine(Y[:m].contiguous(), r, G)
        whole = expert_combine(torch.where((torch.arange(n, device=DEV) < room).unsqueeze(1), Y, torch.zeros_like(Y)), r, G)
        assert torch.equal(V, whole)
        buf = torch.full((room + 3, D), 5.0, dtype=dt, device=DEV)
        dG = torch.empty_like(G)
        _lib.rm_expert_combine_backward(dV.data_ptr(), torch.cat([Y, Y])[:max(room, 1)].contiguous().data_ptr(),
                                        int(dt is torch.bfloat16), r.c, G.data_ptr(), buf.data_ptr(), dG.data_ptr(), room, D,
                                        stream)
        dY, dGw = expert_combine_backward(dV, Y, r, G)
        assert torch.equal(buf[:m], dY[:m]) and (buf[m:] == 5).all()
        assert torch.equal(dG, torch.where(closed > 0, dGw, torch.zeros_like(dGw)))
        q = fp4_expert_gather(X, r, room) if room else None
        if q is not None:
            assert torch.equal(fp4_dequantize(q)[:m], fp4_dequantize(fp4_quantize(expert_gather(X, r)[:n]))[:m])
    ok()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,E", [(3, 2, 5, 4), (8, 4, 768, 8), (70, 3, 1003, 6), (5, 2, 40, 40), (37, 3, 100, 19), (11, 1, 33, 9)])
def test_gather_in_4_bits_is_gather_then_quantize(B, T, D, E, dtype):
    r = expert_sort(gates(B, T, E, 0.5, 9).to(DEV))
    n = r.count()
    X = rows((B, T, D), 10, 2.0).to(DTYPES[dtype]).to(DEV)
    q, want = fp4_expert_gather(X, r, n), fp4_quantize(expert_gather(X, r, n))
    nb = -(-D // 32)
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales[..., :nb], want.scales[..., :nb])
    ok()


# (the last two have more than 2^23 values of experts' outputs)
EXPERTS = [(1, 1, 1, 32, 32), (2, 2, 3, 64, 96), (8, 4, 8, 256, 160), (30, 2, 5, 320, 288), (100, 3, 2, 96, 64),
           (128, 1, 3, 128, 256), (129, 2, 4, 256, 96), (300, 2, 3, 512, 288), (700, 1, 2, 64, 544), (100, 16, 7, 768, 64), (900, 5, 4, 480, 96)]
# hidden layers that fill part of a tile, more than one tile of rows an expert
EXPERTS += [(1500, 2, 3, 32, 32), (1300, 2, 2, 160, 32), (700, 2, 4, 32, 288), (1100, 3, 2, 64, 96)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,E,K,N", EXPERTS + [(40, 2, 3, 1003, 41), (400, 2, 3, 333, 77)])
def test_experts_product(B, T, E, K, N, out):
    G = gates(B, T, E, 0.5, 11)
    G[:, 0, 0] = 0 if E > 1 else 1                   # an expert without rows
    r = expert_sort(G.to(DEV))
    n = r.count()
    from rankmixer_feature_interaction_gb300.api import fp4_quantize_weight
    w = fp4_quantize_weight((torch.randn((T, E, K, N), generator=gen(12)) / K ** 0.5).to(DEV))
    bias = torch.randn((T, E, N), generator=gen(13)).to(DEV)
    x = fp4_expert_gather(rows((B, T, K), 14, 0.5).to(DEV), r)
    y = fp4_expert_matmul(x, w, r, bias, out_dtype=out)
    xv, wv, off = ref.value(x)[:n], ref.weight_value(w), r.offsets.tolist()
    for g in range(T * E):
        a, b = xv[off[g]:off[g + 1]], wv[g // E, g % E]
        if not len(a):
            continue
        want, absolute = a @ b + bias[g // E, g % E], a.abs() @ b.abs() + bias[g // E, g % E].abs()
        tol = ref.sum_bound(K + 1, absolute)
        within(y[off[g]:off[g + 1]], want, tol + (want.abs() + tol) * HALF[out], f"group {g}")
    # room for fewer rows, and nothing written behind the last
    for room in (n // 2, n):
        if room:
            stream = torch.cuda.current_stream().cuda_stream
            buf = torch.full((n + 2, N), 5.0, dtype=y.dtype, device=DEV)
            _lib.rm_fp4_expert_matmul(x.c, w.c, r.c, bias.data_ptr(), buf.data_ptr(), int(out == "bf16"), room, K, N, stream)
            assert torch.equal(buf[:room], y[:room]) and (buf[room:] == 5).all()
    ok()


def moe_reference(m, X, G, b1, b2):
    """(V, bound) in float64 from the 4-bit values, expert by expert."""
    B, T, D = X.shape
    x, w1, w2 = ref.value(fp4_quantize(X)), ref.weight_value(m.W1), ref.weight_value(m.W2)
    V, tol, total = (torch.zeros((B, T, D), dtype=torch.float64, device=DEV) for _ in range(3))
    for t in range(T):
        for e in range(m.E):
            b = torch.nonzero(G[:, t, e] > 0).flatten()
            if b.numel():
                y, d = ref.ffn(x[b, t], w1[t, e], b1[t, e].double(), w2[t, e], b2[t, e].double())
                g = G[b, t, e].double().unsqueeze(1)
                V[b, t] += g * y
                tol[b, t] += g * (d + (y.abs() + d) * ref.HALF_BF16)     # an expert's output in bf16
                total[b, t] += g * (y.abs() + d) * (1 + ref.HALF_BF16)
    return V, tol + ref.sum_bound(m.E, total)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,E,D,F", EXPERTS)
def test_moe(B, T, E, D, F, out):
    w1, b1, w2, b2 = layer((T, E), D, F, 15)
    m = Fp4MoE(w1, b1, w2, b2)
    X = rows((B, T, D), 16, 0.5).to(torch.bfloat16).to(DEV)
    G = gates(B, T, E, 0.4, 17)
    G[0] = 0
    G = G.to(DEV)
    V = m.forward(X, G, out_dtype=out)
    want, tol = moe_reference(m, X, G, b1, b2)
    within(V, want, tol + (want.abs() + tol) * HALF[out], "moe")
    assert (V[0] == 0).all() and torch.equal(V, m.forward(X, G, out_dtype=out))
    # the pieces together give the same
    r = expert_sort(G)
    assert (expert_combine(fp4_expert_matmul(fp4_expert_gather(X, r), m.W1, r, m.b1), r, G) == 0)[0].all()
    ok()


def test_a_training_step_through_the_rows():
    """Rows to their experts, a product there, back with the gates, and the gradients of all of it: as
    the dense sum over experts gives them in float64."""
    B, T, E, D = 60, 3, 4, 48
    g = gen(18)
    G, X = gates(B, T, E, 0.5, 19), torch.randn((B, T, D), generator=g)
    A, C = torch.randn((T * E, D, D), generator=g) / D ** 0.5, torch.randn((B, T, D), generator=g)
    Gd, Xd, Ad = (v.double().requires_grad_() for v in (G, X, A))
    mask = (G > 0).double()
    Vd = torch.einsum("bte,btd,tedf->btf", Gd * mask, Xd, Ad.view(T, E, D, D))
    (Vd * C.double()).sum().backward()
    r = expert_sort(G.to(DEV))
    n, off = r.count(), r.offsets.tolist()
    Xs = expert_gather(X.to(DEV), r, n)
    Y, Ac = torch.empty_like(Xs), A.to(DEV)
    for k in range(T * E):
        Y[off[k]:off[k + 1]] = (Xs[off[k]:off[k + 1]].double() @ Ac[k].double()).float()
    V = expert_combine(Y, r, G.to(DEV))
    dY, dG = expert_combine_backward(C.to(DEV), Y, r, G.to(DEV))
    dXs, dA = torch.empty_like(Xs), torch.zeros_like(Ac)
    for k in range(T * E):
        dXs[off[k]:off[k + 1]] = (dY[off[k]:off[k + 1]].double() @ Ac[k].double().T).float()
        dA[k] = (Xs[off[k]:off[k + 1]].double().T @ dY[off[k]:off[k + 1]].double()).float()
    dX = expert_gather_backward(dXs, r)
    # a handful of float32 roundings (2^-24 each) of sums of at most E D terms, relative to the terms' sizes
    for got, want, size in ((V, Vd, Vd), (dG, Gd.grad, Gd.grad), (dX, Xd.grad, Xd.grad), (dA, Ad.grad, Ad.grad)):
        want = want.detach()
        assert (got.cpu().double() - want).abs().max() <= E * D * 4 * ref.UNIT_F32 * size.detach().abs().max()
    ok()
