"""The router's balance loss, counts and gradient against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from _util import capi, require_cuda
from oracle import balance

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def np64(t):
    return t.detach().double().cpu().numpy()


def inputs(T, E, k, dtype, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed + 1000 * T + E)
    logits = (torch.randn(T, E, generator=g) * std + torch.randn(E, generator=g)).to(dtype)
    idx = torch.rand(T, E, generator=g).topk(k, dim=1).indices.to(torch.int32) if T else torch.zeros(0, k).int()
    return logits, idx


# A share is exp or sigma (2 to 4 ulp: the exponential, the sum 1 + t, the
# reciprocal) over a sum of E terms that adds in a tree of at most 32 per lane
# and five levels, then a product: 48 roundings of 2^-24 cover it.  The fast
# exponential's argument x is rounded when the maximum is subtracted and when
# it is turned to base 2, |x| 2^-24 relative each: shares above 2^-30 have |x|
# up to 21, so 48 more.
EPS_SHARE = 96 * 2.0 ** -24


def check(c, logits, idx, coeff, score, mask=None, off=None, grad=1.25, dev_logits=None):
    T, E = logits.shape
    ref = balance.balance_loss(np64(logits), idx.numpy(), coeff, score, None if mask is None else mask.numpy(),
                               None if off is None else off, grad)
    dl = logits.cuda() if dev_logits is None else dev_logits
    r = c.moe_balance_loss(dl, idx.cuda(), coeff, score=score, token_mask=None if mask is None else mask.cuda(),
                           seq_offsets=None if off is None else torch.tensor(off, dtype=torch.int32).cuda())
    d = c.moe_balance_loss_backward(dl, r, torch.tensor([grad], device="cuda"))
    assert d.dtype == logits.dtype
    assert np.array_equal(r.counts.cpu().numpy(), ref["counts"])
    assert np.array_equal(r.tokens.cpu().numpy(), ref["tokens"])
    assert (np.abs(np64(r.probs) - ref["probs"]) <= EPS_SHARE * ref["probs"] + 2.0 ** -40).all()
    # loss: non-negative terms, each as its share, and one rounding
    assert abs(float(r.loss) - ref["loss"]) <= (EPS_SHARE + 2.0 ** -24) * ref["loss"] + 1e-12 * coeff
    # gradient g p (f - <f, p>) d: p, f, <f, p> (a sum of E) and d are off by
    # EPS_SHARE at most, the difference by that of its two terms
    got, want = np64(d), ref["dlogits"]
    off_ = np.array([0, T]) if off is None else np.asarray(off)
    bound = np.zeros((T, E))
    k = idx.shape[1]
    keep = np.ones(T, bool) if mask is None else mask.numpy().astype(bool)
    p = np.zeros((T, E))
    p[keep] = balance.shares(np64(logits)[keep], score)
    for s in range(len(off_) - 1):
        n = ref["tokens"][s]
        if n == 0:
            continue
        r_ = slice(off_[s], off_[s + 1])
        f = ref["counts"][s] * E / (k * n)
        bound[r_] = 4 * EPS_SHARE * abs(grad) * coeff / (ref["tokens"][-1] * n) * p[r_] * (f + (p[r_] @ f)[:, None])
    fi = torch.finfo(logits.dtype)
    bound = bound + fi.eps / 2 * (np.abs(want) + bound) + fi.smallest_normal * fi.eps + 2.0 ** -40 * coeff / max(T, 1)
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) - bound)
    dead = ~keep
    assert (got[dead] == 0).all()
    return r, d


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 3, 1), (16, 80, 8), (33, 20, 4), (64, 130, 6),
                                   (1000, 128, 8), (257, 256, 8), (100, 300, 3), (70, 512, 8), (40, 1024, 32),
                                   (41, 1023, 2), (9000, 16, 2), (4099, 5, 1)])
def test_matches_oracle(T, E, k, score):
    require_cuda()
    c = capi()
    for name, dt in DTYPES.items():
        logits, idx = inputs(T, E, k, dt)
        check(c, logits, idx, 0.01 if name != "fp16" else 64.0, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("off", [[0, 700], [0, 1, 2, 3, 700], [0, 0, 300, 300, 300, 650, 700, 700], [5, 9, 640],
                                 list(range(0, 701, 4)), list(range(701))])
@pytest.mark.parametrize("T", [700, 200])                 # 16,800 logits take two kernels, 4,800 one
def test_sequences_and_masks(off, score, T):
    require_cuda()
    c = capi()
    logits, idx = inputs(T, 24, 3, torch.float32)
    off = sorted({min(o, T) for o in off}) if len(off) > 100 else [min(o, T) for o in off]
    g = torch.Generator().manual_seed(1)
    check(c, logits, idx, 0.5, score, off=off)
    mask = torch.rand(T, generator=g) < 0.6
    mask[100:180] = False
    check(c, logits, idx, 0.5, score, mask=mask, off=off)
    check(c, logits, idx, 0.5, score, mask=mask.to(torch.uint8), off=off)
    # a mask that leaves nothing: loss 0, gradient 0
    r, d = check(c, logits, idx, 0.5, score, mask=torch.zeros(T, dtype=torch.bool), off=off)
    assert float(r.loss) == 0.0 and int(r.tokens[-1]) == 0 and not d.any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_extreme_logits(score):
    require_cuda()
    c = capi()
    logits, idx = inputs(64, 40, 4, torch.float32)
    logits[:, 7] = -float("inf")                      # an expert masked for everybody
    logits[3] = -float("inf")                         # a token without any expert
    logits[4, 1:] = -float("inf")                     # one expert left
    logits[5] = torch.finfo(torch.float32).min        # masks of the lowest value: all alike
    logits[6, :39] = torch.finfo(torch.float32).min
    logits[7] -= 200.0                                # sigmas that underflow
    logits[8] += 200.0                                # sigmas that are 1
    logits[9] = -70.0 + 20.0 * torch.linspace(-1, 1, 40)
    logits[10] = -58.0 + 20.0 * torch.linspace(-1, 1, 40)
    r, d = check(c, logits, idx, 1.0, score)
    d = d.cpu()
    # (rows 5, 6, 9 and 10 were given new values for expert 7 above)
    assert not d[torch.isneginf(logits)].any() and torch.isneginf(logits[:, 7]).sum() == 60
    assert torch.isfinite(d).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_tokens_may_hold_anything(score):
    require_cuda()
    c = capi()
    logits, idx = inputs(50, 16, 2, torch.bfloat16)
    mask = torch.ones(50, dtype=torch.bool)
    mask[10:20] = False
    dirty = logits.clone()
    dirty[10:15] = float("nan")
    dirty[15:20] = float("inf")
    idx2 = idx.clone()
    idx2[10:20] = 1 << 30
    a = c.moe_balance_loss(logits.cuda(), idx.cuda(), 0.1, score, mask.cuda())
    b = c.moe_balance_loss(dirty.cuda(), idx2.cuda(), 0.1, score, mask.cuda())
    g = torch.ones(1, device="cuda")
    assert torch.equal(a.loss, b.loss) and torch.equal(a.counts, b.counts) and torch.equal(a.probs, b.probs)
    assert torch.equal(c.moe_balance_loss_backward(logits.cuda(), a, g), c.moe_balance_loss_backward(dirty.cuda(), b, g))
    # a NaN in a token that counts shows
    n = c.moe_balance_loss(dirty.cuda(), idx.cuda(), 0.1, score)
    assert torch.isnan(n.loss).all()
    assert torch.isnan(c.moe_balance_loss_backward(dirty.cuda(), n, g)[10]).all()


def test_dropped_choices_and_repeats():
    require_cuda()
    c = capi()
    logits, idx = inputs(40, 12, 4, torch.float32)
    idx[3] = -1
    idx[4] = torch.tensor([12, 5, 5, -2 ** 31])
    idx[5] = 2 ** 31 - 1
    r, _ = check(c, logits, idx, 0.2, "softmax")
    assert int(r.counts.sum()) == 40 * 4 - 4 - 2 - 4


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
def test_strided_logits(dtype, pad):
    require_cuda()
    c = capi()
    logits, idx = inputs(90, 32, 2, DTYPES[dtype])
    big = torch.full((90, 32 + 2 * pad), float("nan"), dtype=DTYPES[dtype], device="cuda")
    big[:, pad:pad + 32] = logits.cuda()
    check(c, logits, idx, 16.0, "sigmoid", dev_logits=big[:, pad:pad + 32])
    # a strided gradient leaves the rest alone
    r = c.moe_balance_loss(logits.cuda(), idx.cuda(), 16.0)
    one = torch.ones(1, device="cuda")
    want = c.moe_balance_loss_backward(logits.cuda(), r, one)
    c.moe_balance_loss_backward(logits.cuda(), r, one, out=big[:, pad:pad + 32])
    assert torch.equal(big[:, pad:pad + 32], want)
    assert torch.isnan(big[:, :pad]).all() and torch.isnan(big[:, pad + 32:]).all()


def test_no_tokens():
    require_cuda()
    c = capi()
    r = c.moe_balance_loss(torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 0.1)
    assert float(r.loss) == 0.0 and not r.counts.any() and r.tokens.tolist() == [0, 0] and not r.probs.any()
    assert c.moe_balance_loss_backward(torch.zeros(0, 8, device="cuda"), r, torch.ones(1, device="cuda")).shape == (0, 8)


def test_gradient_against_differences():
    """Central differences of the kernel's own loss: the fp32 loss is off by
    (EPS_SHARE + 2^-24) loss, divided by 2 h; the truncation is h^2 / 6 times
    a third derivative that is at most a few coeff f / T."""
    require_cuda()
    c = capi()
    T, E, k, coeff, h = 6, 8, 2, 8.0, 0.05
    logits, idx = inputs(T, E, k, torch.float32)
    for score in ("softmax", "sigmoid"):
        lossof = lambda l: float(c.moe_balance_loss(l.cuda(), idx.cuda(), coeff, score).loss)  # noqa: E731
        r = c.moe_balance_loss(logits.cuda(), idx.cuda(), coeff, score)
        d = c.moe_balance_loss_backward(logits.cuda(), r, torch.ones(1, device="cuda")).cpu()
        fmax = float(r.counts.max()) * E / (k * T)
        tol = 2 * EPS_SHARE * float(r.loss) / (2 * h) + h * h / 6 * 8 * coeff * fmax / T
        for t in range(T):
            for e in range(E):
                up, dn = logits.clone(), logits.clone()
                up[t, e] += h
                dn[t, e] -= h
                step = float(up[t, e].double() - dn[t, e].double())
                assert abs((lossof(up) - lossof(dn)) / step - float(d[t, e])) <= tol


def test_same_bits_from_run_to_run_on_streams_and_in_graphs():
    require_cuda()
    c = capi()
    logits, idx = inputs(5000, 96, 6, torch.float32)
    logits, idx = logits.cuda(), idx.cuda()
    off = torch.tensor([0, 100, 100, 4000, 5000], dtype=torch.int32, device="cuda")
    g = torch.full((1,), 0.5, device="cuda")
    a = c.moe_balance_loss(logits, idx, 0.1, seq_offsets=off)
    da = c.moe_balance_loss_backward(logits, a, g)
    ws = torch.empty(c.moe_balance_loss_workspace_size(5000, 96, 4), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            b = c.moe_balance_loss(logits, idx, 0.1, seq_offsets=off, workspace=ws)
            db = c.moe_balance_loss_backward(logits, b, g)
    side.synchronize()
    assert torch.equal(a.loss, b.loss) and torch.equal(a.probs, b.probs) and torch.equal(da, db)
    graphs, outs = [], []
    for _ in range(2):                                 # two graphs share the workspace
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            r = c.moe_balance_loss(logits, idx, 0.1, seq_offsets=off, workspace=ws)
            d = c.moe_balance_loss_backward(logits, r, g)
        graphs.append(gr)
        outs.append((r, d))
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for r, d in outs:
        assert torch.equal(r.loss, a.loss) and torch.equal(r.counts, a.counts) and torch.equal(d, da)


def test_binding_refusals():
    require_cuda()
    c = capi()
    l = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    r = c.moe_balance_loss(l, idx, 0.1)
    one = torch.ones(1, device="cuda")
    for call in (lambda: c.moe_balance_loss(l, idx.long(), 0.1), lambda: c.moe_balance_loss(l, idx[:3], 0.1),
                 lambda: c.moe_balance_loss(l, idx, 0.1, score="relu"), lambda: c.moe_balance_loss(l.t(), idx, 0.1),
                 lambda: c.moe_balance_loss(l, idx, 0.1, token_mask=torch.ones(3, dtype=torch.bool, device="cuda")),
                 lambda: c.moe_balance_loss(l, idx, 0.1, seq_offsets=torch.zeros(1, dtype=torch.int32, device="cuda")),
                 lambda: c.moe_balance_loss_backward(l[:, :7].contiguous(), r, one),
                 lambda: c.moe_balance_loss_backward(l, r, one.double()),
                 lambda: c.moe_balance_loss_backward(l, r, one, out=torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(c.Nvfp4Error):
        c.moe_balance_loss(l, idx, 0.1, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_beside_and_over_the_logits(dtype):
    """Logits and gradient as two column ranges of one buffer give what they
    give apart; a gradient that shares elements with the logits is refused and
    leaves them as they were."""
    require_cuda()
    c = capi()
    T, E = 3000, 24
    logits, idx = inputs(T, E, 3, DTYPES[dtype])
    one = torch.ones(1, device="cuda")
    both = torch.zeros(T + 1, 2 * E, dtype=DTYPES[dtype], device="cuda")
    both[:T, :E] = logits.cuda()
    r = c.moe_balance_loss(both[:T, :E], idx.cuda(), 64.0)
    want = c.moe_balance_loss_backward(logits.cuda(), r, one)
    before = both.clone()
    for out in (both[:T, :E], both[1:, :E], both[:T, E - 4:2 * E - 4], both[:T, 4:E + 4]):
        with pytest.raises(c.Nvfp4Error, match="place"):
            c.moe_balance_loss_backward(both[:T, :E], r, one, out=out)
    assert torch.equal(both, before)
    c.moe_balance_loss_backward(both[:T, :E], r, one, out=both[:T, E:])
    assert torch.equal(both[:T, E:], want) and torch.equal(both[:T, :E], before[:T, :E])


def test_backward_takes_the_forward_calls_length():
    require_cuda()
    c = capi()
    logits, idx = inputs(64, 16, 2, torch.float32)
    r = c.moe_balance_loss(logits.cuda(), idx.cuda(), 0.1)
    one = torch.ones(1, device="cuda")
    assert r.n_tokens == 64
    for other in (logits[:63], torch.cat([logits, logits]), logits[:0]):
        with pytest.raises(ValueError, match="tokens"):
            c.moe_balance_loss_backward(other.cuda(), r, one)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,off", [(200, [0, 90, 200]), (200, [0, 0, 200]), (200, [0, 200, 200]), (200, [0, 0, 0]),
                                   (200, [7, 7, 150]), (200, [200, 200, 200]), (1, [0, 0, 1]), (0, [0, 0, 0]),
                                   (200, [5, 190]), (200, [200, 200]), (682, [0, 300, 682])])
def test_one_kernel_takes_one_or_two_sequences(T, off, score):
    """Up to 16,384 logits in at most two sequences are one kernel's work:
    empty sequences, and masks that empty one of the two or both."""
    require_cuda()
    c = capi()
    logits, idx = inputs(T, 24, 3, torch.float32)
    masks = [None]
    if T:
        for first, last in ((0, T), (off[0], off[1]), (off[-2], off[-1]), (T // 2, T // 2 + 1)):
            m = torch.ones(T, dtype=torch.bool)
            m[first:last] = False
            masks.append(m)
    for m in masks:
        r, d = check(c, logits, idx, 0.5, score, mask=m, off=off)
        if int(r.tokens[-1]) == 0:
            assert float(r.loss) == 0.0 and not r.probs.any() and not r.counts.any() and not d.any()


def test_offsets_past_32_bits():
    """Logits and gradient of more than 2^32 elements: the last tokens, a
    sequence of their own, come out as they do by themselves."""
    require_cuda()
    c = capi()
    T, E, n = 2 ** 25 + 300, 128, 300                          # 8.6 GB of bf16 each
    tail, idx = inputs(n, E, 2, torch.bfloat16)
    logits = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    logits[-n:] = tail.cuda()
    choice = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    choice[-n:] = idx.cuda()
    off = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda")
    g = torch.full((1,), 2.0 ** 10, device="cuda")
    r = c.moe_balance_loss(logits, choice, 1.0, "softmax", seq_offsets=off)
    d = c.moe_balance_loss_backward(logits, r, g)
    alone, d_alone = check(c, tail, idx, 1.0, "softmax", grad=2.0 ** 9)      # one sequence of one, not of two
    assert r.tokens.tolist() == [T - n, n, 2] and int(r.counts[0, 0]) == 2 * (T - n)
    assert torch.equal(r.counts[1:], alone.counts) and torch.equal(d[-n:], d_alone)
    # other pieces, so another order: 300 additions at most, each off by 2^-24
    assert (r.probs[1] - alone.probs[0]).abs().max() <= 300 * 2.0 ** -24 * alone.probs.max()
    # equal shares of 2^-7 add exactly; the mean is one division of two rounded numbers
    assert (r.probs[0] * 128 - 1).abs().max() <= 3 * 2.0 ** -24
    # f is 128 for the one expert that all choose: p (f - <f, p>) = (128 - 1) / 128 there, -1 / 128 elsewhere
    want = torch.full((E,), -1.0 / 128, dtype=torch.float64)
    want[0] = 127.0 / 128
    want *= 2.0 ** 10 / (2 * (T - n))
    for t in (0, 1, T // 2, T - n - 1):
        assert ((d[t].double().cpu() - want).abs() <= (2.0 ** -8 + 8 * 2.0 ** -22) * want.abs()).all()
