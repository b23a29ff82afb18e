"""The MXFP4 and balance-loss operators together, as a user's program calls
them: a routed-expert layer built from moe_route's rows, and one training step
of a projection behind a router."""
import numpy as np
import pytest
import torch

from _util import capi, require_cuda
from oracle import balance, mxfp4

pytestmark = pytest.mark.gpu


def np64(t):
    return t.detach().double().cpu().numpy()


def mx(x):
    """x's MXFP4 values in float64."""
    return mxfp4.dequantize(*mxfp4.quantize(x), x.shape[1])


@pytest.mark.parametrize("T", [1, 16, 700])
def test_routed_experts_from_the_parts(T):
    """route -> counts and loss -> gathered gate/up -> SiLU * up -> down with
    the routing weights -> combine, against the same steps in 64 bits on the
    routing that moe_route chose."""
    require_cuda()
    c = capi()
    E, H, I, k = 8, 256, 128, 2
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, H, generator=g).bfloat16()
    wr = (torch.randn(E, H, generator=g) * 0.05).bfloat16()
    bias = torch.randn(E, generator=g) * 0.01
    gate_up = (torch.randn(E, 2 * I, H, generator=g) * 0.05).bfloat16()
    down = (torch.randn(E, H, I, generator=g) * 0.05).bfloat16()
    xd = x.cuda()
    wgu, wdn = c.mxfp4_quantize(gate_up.cuda()), c.mxfp4_quantize(down.cuda())
    r = c.moe_route(xd, wr.cuda(), bias.cuda(), k, 2.5)
    b = c.moe_balance_loss(r["logits"], r["topk_idx"], 0.01)
    off = r["expert_offsets"]
    counts = b.counts[0]
    gu = c.mxfp4_linear(xd, wgu, out_dtype=torch.float32, perm=r["perm"], expert_offsets=off, expert_counts=counts)
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    cap = r["perm"].numel()
    row_w = torch.zeros(cap, device="cuda")
    row_w[r["inv_perm"].reshape(-1).long()] = r["topk_w"].reshape(-1)
    y = c.mxfp4_linear(h, wdn, expert_offsets=off, expert_counts=counts, row_weight=row_w, out_dtype=torch.float32)
    out = y[r["inv_perm"].long()].sum(dim=1)

    idx, w = r["topk_idx"].cpu().numpy(), np64(r["topk_w"])
    ref = balance.balance_loss(np64(r["logits"]), idx, 0.01, "sigmoid")
    assert np.array_equal(counts.cpu().numpy(), ref["counts"][0]) and abs(float(b.loss) - ref["loss"]) <= 1e-5 * ref["loss"]
    xq = mx(x.double().numpy())
    gq = mx(gate_up.double().numpy().reshape(E * 2 * I, H)).reshape(E, 2 * I, H)
    dq = mx(down.double().numpy().reshape(E * H, I)).reshape(E, H, I)
    # the intermediate is quantised from the device's h, whose codes may differ
    # from an exact h's where that lies next to a rounding border
    hd = mx(np64(h[r["inv_perm"].reshape(-1).long()])).reshape(T, k, I)
    want = np.zeros((T, H))
    bound = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            z = gq[e] @ xq[t]
            exact_h = z[:I] / (1 + np.exp(-z[:I])) * z[I:]
            got_h = np64(h[int(r["inv_perm"][t, j])])
            # fp32 sums of H products, then SiLU and a product in fp32
            mag = np.abs(gq[e]) @ np.abs(xq[t])
            slack = (H + 2) * 2.0 ** -23 * mag
            tol = 1.2 * slack[:I] * np.abs(z[I:]) + slack[I:] * np.abs(z[:I]) + 1e-5 * np.abs(exact_h) + 1e-7
            assert (np.abs(got_h - exact_h) <= tol).all()
            want[t] += w[t, j] * (dq[e] @ hd[t, j])
            bound[t] += w[t, j] * (I + k + 4) * 2.0 ** -23 * (np.abs(dq[e]) @ np.abs(hd[t, j]))
    assert (np.abs(np64(out) - want) <= bound + 1e-9).all()


def test_training_step_of_a_projection_behind_a_router():
    """Forward, both gradients of an MXFP4 projection, and the balance loss's
    gradient, captured into one graph that is replayed after its inputs have
    changed; each output against its formula."""
    require_cuda()
    c = capi()
    T, H, N, E, k = 300, 384, 200, 16, 3
    g = torch.Generator().manual_seed(0)
    draw = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w, dy = draw(T, H).bfloat16().cuda(), (draw(N, H) * 0.1).bfloat16().cuda(), draw(T, N).bfloat16().cuda()
    logits = draw(T, E).cuda()
    idx = logits.topk(k).indices.int()
    off = torch.tensor([0, 90, 250], dtype=torch.int32, device="cuda")        # the last 50 tokens are padding
    scale = torch.full((1,), 128.0, device="cuda")

    def step():
        y = c.mxfp4_linear(x, c.mxfp4_quantize(w), out_dtype=torch.float32)
        dx = c.mxfp4_matmul(c.mxfp4_quantize(dy), c.mxfp4_quantize_transposed(w), out_dtype=torch.float32)
        dw = c.mxfp4_matmul(c.mxfp4_quantize_transposed(dy), c.mxfp4_quantize_transposed(x), out_dtype=torch.float32)
        b = c.moe_balance_loss(logits, idx, 0.01, score="softmax", seq_offsets=off)
        return y, dx, dw, b.loss, c.moe_balance_loss_backward(logits, b, scale)

    eager = step()                                                  # stays alive through the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, eager))
    for t in (x, w, dy, logits):
        t.copy_(torch.roll(t, 1, 0))
    idx.copy_(logits.topk(k).indices.int())
    graph.replay()
    torch.cuda.synchronize()
    y, dx, dw, loss, dl = (np64(t) for t in outs)
    xn, wn, dyn = np64(x), np64(w), np64(dy)

    def close(got, a, b):
        assert (np.abs(got - a @ b.T) <= (a.shape[1] + 1) * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T) + 1e-30).all()
    close(y, mx(xn), mx(wn))
    close(dx, mx(dyn), mx(wn.T))
    close(dw, mx(dyn.T), mx(xn.T))
    ref = balance.balance_loss(np64(logits), idx.cpu().numpy(), 0.01, "softmax", None, off.cpu().numpy(), 128.0)
    assert abs(float(loss[0]) - ref["loss"]) <= 1e-5 * ref["loss"]
    assert np.abs(dl - ref["dlogits"]).max() <= 4e-5 * np.abs(ref["dlogits"]).max()
    assert (dl[250:] == 0).all()


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("offsets", [None, [0, 40, 40, 300], [10, 200, 290]])
def test_routed_rows_beside_a_loss_that_leaves_tokens_out(masked, offsets):
    """Every routed row is multiplied: with the loss's counts summed over the
    sequences where it keeps every token, else without counts."""
    require_cuda()
    c = capi()
    T, E, H, N, k = 300, 8, 256, 128, 2
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, H, generator=g).bfloat16()
    w = (torch.randn(E, N, H, generator=g) * 0.05).bfloat16()
    r = c.moe_route(x.cuda(), (torch.randn(E, H, generator=g) * 0.05).bfloat16().cuda(), torch.zeros(E, device="cuda"),
                    k, 2.5)
    mask = (torch.rand(T, generator=g) < 0.7).cuda() if masked else None
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    b = c.moe_balance_loss(r["logits"], r["topk_idx"], 0.01, token_mask=mask, seq_offsets=off)
    counts = b.counts.sum(0, dtype=torch.int32)
    keeps_all = not masked and (offsets is None or offsets[0] == 0)
    assert (int(counts.sum()) == T * k) == keeps_all
    out = c.mxfp4_linear(x.cuda(), c.mxfp4_quantize(w.cuda()), perm=r["perm"], expert_offsets=r["expert_offsets"],
                         expert_counts=counts if keeps_all else None, out_dtype=torch.float32)
    xq, wq = mx(x.double().numpy()), mx(w.double().numpy().reshape(E * N, H)).reshape(E, N, H)
    idx, got = r["topk_idx"].cpu().numpy(), np64(out[r["inv_perm"].long()])
    for t in range(T):
        for j in range(k):
            m = wq[idx[t, j]]
            # fp32 sums of H products, each addition truncated at most
            assert (np.abs(got[t, j] - m @ xq[t]) <= (H + 2) * 2.0 ** -23 * (np.abs(m) @ np.abs(xq[t])) + 1e-30).all()
    rest = torch.ones(out.shape[0], dtype=torch.bool)
    rest[r["inv_perm"].reshape(-1).long().cpu()] = False
    assert not out[rest.cuda()].any()
