"""The operators over vocabulary-parallel logits against the 64-bit oracle.

Tolerances, derived from the arithmetic (u = 2^-24):
- a term 2^d, d = (x - m) c <= 0: the argument is off by at most 3 u |d|, the
  exponential by 2^-22; weighted with the terms themselves (2^d |d| < 0.54) a
  sum of them is off by less than 2^-21 of itself. Adding n positive terms in
  any order whose longest chain is n / 64 + 64 additions adds that many u. So
  log(sum) is off by at most E = 2^-20 + (n / 64 + 64) u.
- a log probability lp = (x - m) / T - log(sum): E + 4 u (|lp| + E).
- the entropy log(sum) - u / s / T: E + 2 E |u / s| / T, and |u / s| / T is at
  most log n plus the entropy: E (1 + 4 log n).
- a probability from lp: relative 2^-22 + the error of lp + 3 u |lp| = R;
  a gradient: p (|a| + |b| (|lp| + |h|)) R + p |b| (error of lp and of h)
  + 4 u |a| at the token, plus terms below 2^-126 flushed to zero.
- a teacher's q: R with the largest |t / T| in place of |lp| (twice: the
  entry's own and the one in the log-sum), and K u.
A bf16 gradient is rounded once more: it has to lie between the roundings of
the two ends of its interval."""
import numpy as np
import pytest
import torch

import collective_communication_planner_gb300 as tccl
from oracle import vocab as vo

pytestmark = pytest.mark.gpu
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def groups():
    made = {}

    def get(p):
        if p not in made:
            made[p] = tccl.Group(p)
        return made[p]

    yield get
    for g in made.values():
        g.close()


# ------------------------------------------------------------- tolerances
def tol_sum(n):
    return 2.0 ** -20 + (n / 64 + 64) * U


def tol_lp(lp, n):
    lp = np.where(np.isfinite(lp), lp, 0.0)
    return tol_sum(n) + 4 * U * (np.abs(lp) + tol_sum(n))


def tol_entropy(n):
    return tol_sum(n) * (1 + 4 * np.log(max(n, 2)))


def tol_p(lp, n):
    return 2.0 ** -22 + tol_lp(lp, n) + 3 * U * np.abs(np.where(np.isfinite(lp), lp, 0.0))


def close(got, exp, tol, what):
    got = np.asarray(got, dtype=np.float64)
    # past the largest fp32 number the nearest result is infinite
    exp = np.where(np.abs(exp) > np.finfo(np.float32).max, np.copysign(np.inf, exp), exp)
    fin = np.isfinite(exp)
    same = np.where(np.isnan(exp), np.isnan(got), got == exp)
    assert np.all(same[~fin]), f"{what}: special values differ"
    tol = np.broadcast_to(tol, exp.shape)
    err = np.abs(got[fin] - exp[fin])
    assert np.all(err <= tol[fin]), f"{what}: error {np.max(err - tol[fin])} above the bound"


def close_grad(got, exp, tol, dtype, what):
    tol = tol + 2.0 ** -120
    if dtype == "bf16":
        # rounding is monotone, so a value within tol of exp rounds into [lo, hi]
        fin = np.isfinite(exp)
        lo, hi = (torch.from_numpy(np.where(fin, exp + s * tol, 0.0)).bfloat16().double().numpy() for s in (-1, 1))
        inside = (got >= lo) & (got <= hi)
        assert np.all(inside[fin]), f"{what}: {np.count_nonzero(~inside[fin])} values outside their interval"
        tol = np.where(fin, np.abs(got - exp), 0.0)
    close(got, exp, tol, what)


# ------------------------------------------------------------- inputs
def make_logits(rng, rows, vocab, dtype, sharp=True):
    """[rows, vocab] on the host, already rounded to the datatype."""
    x = rng.normal(size=(rows, vocab)) * 2 + rng.normal(size=(rows, 1)) * 4
    if sharp and vocab > 4:
        x[np.arange(rows), rng.integers(0, vocab, rows)] += rng.uniform(0, 12, rows)
    return torch.from_numpy(x).to(TORCH[dtype])


def cut(x, p, shard, gap=0, offset=0, fill=float("nan")):
    """The matrix as p ranks hold it: columns by blocks of `shard`, rows
    shard + gap apart, each buffer `offset` elements into its allocation;
    padding columns and gaps hold `fill`."""
    rows, vocab = x.shape
    out = []
    for r in range(p):
        raw = torch.full((rows * (shard + gap) + offset,), fill, dtype=x.dtype, device="cuda")
        m = raw[offset:].view(rows, shard + gap)[:, :shard]
        lo, hi = min(r * shard, vocab), min((r + 1) * shard, vocab)
        m[:, :hi - lo] = x[:, lo:hi].cuda()
        out.append(m)
    return out


def glue(mats, vocab):
    """(valid columns, padding columns) of per-rank matrices, in fp64 on the host."""
    whole = torch.cat([m.double() for m in mats], 1).cpu().numpy()
    return whole[:, :vocab], whole[:, vocab:]


def f32(*shape):
    return torch.full(shape, 777.0, dtype=torch.float32, device="cuda")


def dev(a, dtype=torch.float32):
    return torch.as_tensor(np.asarray(a)).to(dtype).cuda()


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------- checked calls
def check_log_probs(g, x, p, shard, tokens, dtype, temperature=1.0, k=0, gap=0, offset=0, cap=0,
                    logits=None):
    rows, vocab = x.shape
    logits = cut(x, p, shard, gap, offset) if logits is None else logits
    lp, ent, st = f32(rows), f32(rows), f32(rows, 2)
    top, ids = (f32(rows, k), torch.full((rows, k), -7, device="cuda")) if k else (None, None)
    tok = None if tokens is None else dev(tokens, torch.int64)
    g.log_probs(logits, tok, None if tokens is None else lp, ent, st, top, ids, vocab=vocab,
                temperature=temperature, cta_cap=cap)
    torch.cuda.synchronize()
    assert g.query_error() == tccl.tcclSuccess
    e = vo.log_probs(x.double().numpy(), tokens, temperature, k)
    if tokens is not None:
        close(host(lp), e["log_probs"], tol_lp(e["log_probs"], vocab), "log_probs")
    close(host(ent), e["entropy"], tol_entropy(vocab), "entropy")
    got = host(st)
    close(got[:, 0], e["stats"][:, 0], 0.0, "stats maximum")
    close(got[:, 1], e["stats"][:, 1], tol_sum(vocab) + U * np.log(max(vocab, 2)), "stats sum")
    if k:
        assert np.array_equal(ids.cpu().numpy(), e["top_ids"]), "top_ids"
        close(host(top), e["top_log_probs"], tol_lp(e["top_log_probs"], vocab), "top_log_probs")
    return lp, ent, st, top, ids


def stats_of(x, temperature):
    _, m, s = vo.log_softmax(x.double().numpy(), temperature)
    return dev(np.stack([m, s], 1))


def grad_buffers(x, p, shard, gap, offset):
    return cut(torch.full(x.shape, 5.0, dtype=x.dtype), p, shard, gap, offset, fill=5.0)


def check_grads(grads, exp, tol, dtype, vocab, what):
    got, pad = glue(grads, vocab)
    assert not pad.any(), f"{what}: padding columns are not zero"
    close_grad(got, exp, tol, dtype, what)


def check_backward(g, x, p, shard, tokens, dtype, a, b, temperature=1.0, gap=0, gap_out=0, offset=0,
                   offset_out=0, cap=0, in_place=False):
    rows, vocab = x.shape
    logits = cut(x, p, shard, gap, offset)
    grads = logits if in_place else grad_buffers(x, p, shard, gap_out, offset_out)
    lp, _, _ = vo.log_softmax(x.double().numpy(), temperature)
    h = vo.entropy(lp)
    g.log_probs_backward(logits, dev(tokens, torch.int64), stats_of(x, temperature), dev(a), grads,
                         entropy=None if b is None else dev(h),
                         d_entropy=None if b is None else dev(b), vocab=vocab,
                         temperature=temperature, cta_cap=cap)
    torch.cuda.synchronize()
    assert g.query_error() == tccl.tcclSuccess
    exp = vo.log_probs_backward(x.double().numpy(), tokens, temperature, a, b)
    A, B = np.abs(a)[:, None], 0.0 if b is None else np.abs(b)[:, None]
    L = np.abs(np.where(np.isfinite(lp), lp, 0.0))
    H = np.abs(np.where(np.isfinite(h), h, 0.0))[:, None]
    P = np.exp(np.where(np.isnan(lp), 0.0, lp))
    hot = np.zeros(x.shape)
    ok = (tokens >= 0) & (tokens < vocab)
    hot[ok, tokens[ok]] = 1.0
    tol = (P * (A + B * (L + H)) * (tol_p(lp, vocab) + 8 * U)
           + P * B * (tol_lp(lp, vocab) + 4 * U * H) + 4 * U * A * hot) / temperature
    check_grads(grads, exp, tol, dtype, vocab, "log_probs_backward")
    return grads


def tol_teacher(t, temperature, k):
    big = np.abs(np.where(np.isfinite(t), t, 0.0)).max(axis=1, keepdims=True) / temperature
    return 2.0 ** -21 + 8 * U * (1 + 2 * big) + k * U


def distill_bounds(x, ids, t, temperature, lse, w):
    rows, vocab = x.shape
    xd = x.double().numpy()
    lp, _, _ = vo.log_softmax(xd, temperature)
    q, log_q = vo.teacher(ids, t, temperature, lse, vocab)
    loss, g = vo.distill(xd, ids, t, temperature, lse, w)
    if lse is not None:
        t = np.concatenate([t, np.asarray(lse)[:, None] * temperature], 1)
    rq = tol_teacher(t, temperature, ids.shape[1])
    picked = np.take_along_axis(lp, np.clip(ids, 0, vocab - 1), 1)
    size = np.abs(np.where(q > 0, log_q, 0.0)) + np.abs(np.where(np.isfinite(picked), picked, 0.0))
    tl = (q * (size * (rq + 8 * U) + rq + tol_lp(picked, vocab))).sum(1)
    tg = None
    if w is not None:
        P = np.exp(np.where(np.isnan(lp), 0.0, lp))
        Q = np.nansum(q, 1, keepdims=True)
        at = np.zeros(x.shape)
        for i in range(rows):
            on = q[i] > 0
            np.add.at(at[i], ids[i][on], q[i][on])
        tg = (np.abs(w)[:, None] / temperature) * (Q * P * (tol_p(lp, vocab) + rq + 4 * U) + at * (rq + 4 * U))
    return loss, tl, g, tg


def check_distill(g, x, p, shard, ids, t, dtype, temperature=1.0, lse=None, w=None, teacher="f32",
                  gap=0, gap_out=0, offset=0, offset_out=0, cap=0, in_place=False, ways=("step", "apart")):
    """The loss with its gradient in one call ("step"), and the forward and the
    gradient as two calls ("apart")."""
    rows, vocab = x.shape
    tt = torch.from_numpy(t).to(TORCH[teacher])
    loss, tl, grad, tg = distill_bounds(x, ids, tt.double().numpy(), temperature, lse, w)
    kw = dict(vocab=vocab, temperature=temperature, cta_cap=cap,
              teacher_lse=None if lse is None else dev(lse))
    outs = []
    for way in ways:
        logits = cut(x, p, shard, gap, offset)
        grads = None if w is None else logits if in_place else grad_buffers(x, p, shard, gap_out, offset_out)
        got, st = f32(rows), f32(rows, 2)
        if way == "step":
            g.distill(logits, dev(ids, torch.int64), tt.cuda(), got, st,
                      weights=None if w is None else dev(w), grads=grads, **kw)
        else:
            g.distill(logits, dev(ids, torch.int64), tt.cuda(), got, st, **kw)
            if w is not None:
                g.distill_backward(logits, dev(ids, torch.int64), tt.cuda(), st, dev(w), grads, **kw)
        torch.cuda.synchronize()
        assert g.query_error() == tccl.tcclSuccess
        close(host(got), loss, tl, f"loss ({way})")
        _, m, s = vo.log_softmax(x.double().numpy(), temperature)
        close(host(st)[:, 0], m, 0.0, "stats maximum")
        close(host(st)[:, 1], s, tol_sum(vocab) + U * np.log(max(vocab, 2)), "stats sum")
        if w is not None:
            check_grads(grads, grad, tg, dtype, vocab, f"distill gradient ({way})")
        outs.append((got, st, grads))
    return outs


def make_teacher(rng, rows, vocab, k):
    """Distinct ids where the vocabulary has as many, a few entries empty."""
    ids = np.stack([rng.permutation(max(vocab, k))[:k] for _ in range(rows)])
    ids = np.where(ids < vocab, ids, -1)
    ids[rng.random(ids.shape) < 0.1] = -1
    return ids, rng.normal(size=(rows, k)) * 3


# rows, vocab, ranks, shard: one column, less than a vector, odd shards, ranks
# without a column, whole vectors, many ranks, more columns than one pass holds
SHAPES = [(1, 1, 1, 1), (3, 5, 2, 3), (2, 7, 4, 3), (5, 64, 1, 64), (4, 1000, 3, 334),
          (3, 1000, 8, 128), (2, 4099, 64, 65), (7, 8192, 8, 1024), (2, 33000, 5, 6600),
          (1, 70001, 3, 23334), (170, 515, 2, 258), (2, 50257, 1, 50304)]
DTYPES = ["f32", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,p,shard", SHAPES)
def test_log_probs(groups, dtype, rows, vocab, p, shard):
    rng = np.random.default_rng(rows * 131 + vocab)
    x = make_logits(rng, rows, vocab, dtype)
    tokens = rng.integers(0, vocab, rows)
    for k, temperature in ((0, 1.0), (1, 0.7), (20, 2.0), (128, 1.0)):
        check_log_probs(groups(p), x, p, shard, tokens, dtype, temperature, k)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,p,shard", SHAPES)
def test_log_probs_backward(groups, dtype, rows, vocab, p, shard):
    rng = np.random.default_rng(rows * 137 + vocab)
    x = make_logits(rng, rows, vocab, dtype)
    tokens = rng.integers(0, vocab, rows)
    a, b = rng.normal(size=rows).astype(np.float32), rng.normal(size=rows).astype(np.float32)
    for bb, temperature in ((None, 1.0), (b, 0.7)):
        check_backward(groups(p), x, p, shard, tokens, dtype, a, bb, temperature)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,p,shard", SHAPES)
def test_distill(groups, dtype, rows, vocab, p, shard):
    rng = np.random.default_rng(rows * 139 + vocab)
    x = make_logits(rng, rows, vocab, dtype)
    w = rng.normal(size=rows).astype(np.float32)
    for k, temperature, known, teacher in ((1, 1.0, False, "f32"), (17, 0.7, True, "bf16"),
                                           (128, 2.0, False, "bf16")):
        ids, t = make_teacher(rng, rows, vocab, k)
        lse = (rng.normal(size=rows) + 4).astype(np.float32) if known else None
        check_distill(groups(p), x, p, shard, ids, t, dtype, temperature, lse, w, teacher)


# every pair of source and destination alignment that 16-byte accesses can meet
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("gap,offset,gap_out,offset_out",
                         [(0, 0, 0, 0), (8, 0, 0, 0), (8, 8, 8, 8), (1, 0, 0, 0), (0, 1, 0, 0),
                          (0, 0, 3, 0), (0, 0, 0, 5), (3, 2, 5, 7), (4, 4, 2, 6), (7, 7, 7, 7)])
def test_strides_and_alignment(groups, dtype, gap, offset, gap_out, offset_out):
    rng = np.random.default_rng(gap * 8 + offset)
    for p, shard, vocab in ((3, 720, 2001), (2, 1537, 3070)):
        rows = 5
        x = make_logits(rng, rows, vocab, dtype)
        tokens = np.array([0, vocab - 1, shard - 1, shard, -1])
        a, b = rng.normal(size=rows).astype(np.float32), rng.normal(size=rows).astype(np.float32)
        kw = dict(gap=gap, offset=offset)
        check_log_probs(groups(p), x, p, shard, tokens, dtype, k=9, **kw)
        kw.update(gap_out=gap_out, offset_out=offset_out)
        check_backward(groups(p), x, p, shard, tokens, dtype, a, b, **kw)
        ids, t = make_teacher(rng, rows, vocab, 12)
        ids[0, :4] = [0, shard - 1, shard, vocab - 1]
        check_distill(groups(p), x, p, shard, ids, t, dtype, w=a, **kw)


def test_ranks_of_different_alignment(groups):
    """Rank buffers that start at different addresses mod 16."""
    rng = np.random.default_rng(3)
    rows, vocab, p, shard = 4, 2900, 3, 968
    for dtype in DTYPES:
        x = make_logits(rng, rows, vocab, dtype)
        parts = [cut(x, p, shard, 0, off)[r] for r, off in enumerate((0, 3, 1))]
        tokens = np.array([5, 1000, 2000, 2899])
        check_log_probs(groups(p), x, p, shard, tokens, dtype, k=6, logits=parts)
        a = rng.normal(size=rows).astype(np.float32)
        outs = [grad_buffers(x, p, shard, 0, off)[r] for r, off in enumerate((2, 0, 3))]
        groups(p).log_probs_backward(parts, dev(tokens, torch.int64), stats_of(x, 1.0), dev(a), outs, vocab=vocab)
        lp, _, _ = vo.log_softmax(x.double().numpy(), 1.0)
        exp = vo.log_probs_backward(x.double().numpy(), tokens, 1.0, a, None)
        tol = np.abs(a)[:, None] * (np.exp(lp) * (tol_p(lp, vocab) + 8 * U) + 4 * U)
        check_grads(outs, exp, tol, dtype, vocab, "grads")


def test_column_blocks_of_one_matrix(groups):
    """Per-rank views into one [rows, vocab] matrix: in place, and into the
    column blocks of another matrix."""
    rng = np.random.default_rng(4)
    rows, p, shard = 6, 4, 520
    vocab = p * shard
    x = make_logits(rng, rows, vocab, "bf16")
    a = rng.normal(size=rows).astype(np.float32)
    tokens = rng.integers(0, vocab, rows)
    lp, _, _ = vo.log_softmax(x.double().numpy(), 1.0)
    exp = vo.log_probs_backward(x.double().numpy(), tokens, 1.0, a, None)
    tol = np.abs(a)[:, None] * (np.exp(lp) * (tol_p(lp, vocab) + 8 * U) + 4 * U)
    whole = x.cuda()
    blocks = lambda m: [m[:, r * shard:(r + 1) * shard] for r in range(p)]
    check_log_probs(groups(p), x, p, shard, tokens, "bf16", k=5, logits=blocks(whole))
    for target in (torch.empty_like(whole), whole):
        groups(p).log_probs_backward(blocks(whole), dev(tokens, torch.int64), stats_of(x, 1.0), dev(a), blocks(target))
        check_grads(blocks(target), exp, tol, "bf16", vocab, "grads")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,p,shard", [(1000, 3, 334), (8192, 8, 1024), (40000, 2, 20000)])
def test_in_place(groups, dtype, vocab, p, shard):
    rng = np.random.default_rng(vocab)
    rows = 9
    x = make_logits(rng, rows, vocab, dtype)
    a, b = rng.normal(size=rows).astype(np.float32), rng.normal(size=rows).astype(np.float32)
    tokens = rng.integers(0, vocab, rows)
    check_backward(groups(p), x, p, shard, tokens, dtype, a, b, in_place=True)
    ids, t = make_teacher(rng, rows, vocab, 33)
    check_distill(groups(p), x, p, shard, ids, t, dtype, w=a, in_place=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,p,shard", [(900, 3, 300), (9000, 4, 2256)])
def test_masked_logits(groups, dtype, vocab, p, shard):
    """-inf and the type's lowest value in masked places, rows that the mask
    leaves nothing or little of."""
    rng = np.random.default_rng(17)
    rows = 12
    lowest = torch.finfo(TORCH[dtype]).min
    x = make_logits(rng, rows, vocab, dtype)
    inf = float("inf")
    x[0] = -inf
    x[1] = -inf
    x[1, vocab // 2] = 3.0
    x[2] = lowest                      # uniform
    x[3] = lowest
    x[3, 7] = -2.0
    x[4] = -inf
    x[4, 5:9] = lowest                 # uniform over four columns
    x[5, : vocab // 2] = -inf
    x[6, vocab // 2:] = lowest
    x[7] = -inf
    x[7, [1, vocab - 1, 400]] = torch.tensor([1.0, 2.0, 2.0]).to(x.dtype)
    x[8] = 0.0                         # all equal
    x[9] = -0.0
    x[9, 11:15] = 0.0                  # zeros of either sign are equal
    x[10] = -30000.0                   # a large common offset
    x[10, 3] = -29990.0
    x[11] += 10000.0
    tokens = np.array([4, vocab // 2, 3, 7, 6, vocab - 1, 3, 1, 2, 12, 3, 8])
    for k in (0, 5, 128):
        check_log_probs(groups(p), x, p, shard, tokens, dtype, k=k)
    # masked tokens, on other columns than the ones left
    check_log_probs(groups(p), x, p, shard, (tokens + 1) % vocab, dtype, temperature=0.5, k=3)
    a, b = rng.normal(size=rows).astype(np.float32), rng.normal(size=rows).astype(np.float32)
    check_backward(groups(p), x, p, shard, tokens, dtype, a, b)
    check_backward(groups(p), x, p, shard, tokens, dtype, a, None, temperature=0.5)
    ids = np.stack([rng.permutation(vocab)[:6] for _ in range(rows)])
    t = rng.normal(size=(rows, 6))
    for i in range(rows):  # the teacher on columns that are left, where there are any
        ok = np.flatnonzero(np.isfinite(x[i].double().numpy()) & (x[i].double().numpy() > -1e30))
        if len(ok):
            ids[i] = ok[np.arange(6) % len(ok)]
            ids[i, len(ok):] = -1
    check_distill(groups(p), x, p, shard, ids, t, dtype, w=a)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinity(groups, dtype):
    rng = np.random.default_rng(18)
    p, shard, vocab, rows = 2, 1030, 2050, 5
    x = make_logits(rng, rows, vocab, dtype)
    x[0, 1500] = float("nan")
    x[1, 3] = float("inf")
    x[2, 0], x[2, 2049] = float("nan"), float("inf")
    tokens = np.array([3, 3, 9, 4, 5])
    logits = cut(x, p, shard)
    lp, ent, st = f32(rows), f32(rows), f32(rows, 2)
    top, ids = f32(rows, 4), torch.zeros(rows, 4, dtype=torch.int64, device="cuda")
    groups(p).log_probs(logits, dev(tokens, torch.int64), lp, ent, st, top, ids, vocab=vocab)
    for t in (lp, ent, st[:, 1], top[:, 0]):
        assert torch.isnan(t[:3]).all() and torch.isfinite(t[3:]).all()
    assert (ids[:3] == -1).all() and (ids[3:] >= 0).all()
    grads = grad_buffers(x, p, shard, 0, 0)
    ones = dev(np.ones(rows))
    groups(p).log_probs_backward(logits, dev(tokens, torch.int64), st, ones, grads, entropy=ent, d_entropy=ones, vocab=vocab)
    got, pad = glue(grads, vocab)
    assert np.isnan(got[:3]).all() and np.isfinite(got[3:]).all() and not pad.any()
    tid = dev(np.tile([1, 2, 3], (rows, 1)), torch.int64)
    for fused in (True, False):
        loss, st2, grads = f32(rows), f32(rows, 2), grad_buffers(x, p, shard, 0, 0)
        tz = f32(rows, 3)
        if fused:
            groups(p).distill(logits, tid, tz, loss, st2, weights=ones, grads=grads, vocab=vocab)
        else:
            groups(p).distill(logits, tid, tz, loss, st2, vocab=vocab)
            groups(p).distill_backward(logits, tid, tz, st2, ones, grads, vocab=vocab)
        got, pad = glue(grads, vocab)
        assert torch.isnan(loss[:3]).all() and torch.isfinite(loss[3:]).all()
        assert np.isnan(got[:3]).all() and np.isfinite(got[3:]).all() and not pad.any()


def test_unscored_rows(groups):
    rng = np.random.default_rng(19)
    p, shard, vocab, rows = 4, 256, 1000, 7
    x = make_logits(rng, rows, vocab, "bf16")
    x[1] = float("nan")  # not read
    tokens = np.array([0, -1, vocab, 999, -100, 1 << 40, 256])
    check_log_probs(groups(p), x, p, shard, tokens, "bf16", k=3)
    a, b = rng.normal(size=rows).astype(np.float32), rng.normal(size=rows).astype(np.float32)
    a[3] = b[3] = 0.0
    check_backward(groups(p), x, p, shard, tokens, "bf16", a, b)
    x[1] = 0.0
    check_log_probs(groups(p), x, p, shard, None, "bf16", k=3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_alternatives_in_every_order(groups, dtype):
    """Values that rise, fall, repeat, or crowd into one place of the row: the
    selection meets every amount of ties and every position."""
    p, shard, vocab = 3, 5000, 14990
    rng = np.random.default_rng(20)
    j = np.arange(vocab)
    rows = [j * 1e-3, -j * 1e-3, (j % 7) * 1.0, (j // 100) * 1.0, np.zeros(vocab), (j == 9000) * 5.0,
            np.where(j % 2048 < 8, 5.0, rng.normal(size=vocab)),
            np.where((j >= 4000) & (j < 6100), 3.0 + (j % 5), rng.normal(size=vocab)),
            np.round(rng.normal(size=vocab) * 2) / 2, np.minimum(rng.normal(size=vocab), 1.0)]
    x = torch.from_numpy(np.stack(rows)).to(TORCH[dtype])
    for k in (1, 2, 31, 32, 33, 100, 128):
        check_log_probs(groups(p), x, p, shard, None, dtype, k=k)


@pytest.mark.parametrize("dtype", DTYPES)
def test_teacher_entries(groups, dtype):
    """Columns named twice or more, empty entries, -inf and masked columns."""
    rng = np.random.default_rng(21)
    p, shard, vocab, rows, k = 2, 600, 1190, 6, 40
    x = make_logits(rng, rows, vocab, dtype)
    ids, t = make_teacher(rng, rows, vocab, k)
    ids[0] = 77
    ids[1, ::2] = 601
    ids[2] = -1
    t[3] = -np.inf
    t[4, 1:] = -np.inf
    ids[4, 0] = 5
    ids[5, 3] = 1190  # a padding column is no column
    w = rng.normal(size=rows).astype(np.float32)
    w[1] = 0.0
    check_distill(groups(p), x, p, shard, ids, t, dtype, w=w)
    lse = np.full(rows, 3.0, dtype=np.float32)
    check_distill(groups(p), x, p, shard, ids, t, dtype, temperature=1.5, lse=lse, w=w, teacher="bf16")
    x[0, 77] = float("-inf")  # the student gives 0 where the teacher does not: loss +inf
    check_distill(groups(p), x, p, shard, ids, t, dtype, w=w)


@pytest.mark.parametrize("cap", [1, 3, 16, 40])
def test_caps_and_many_rows(groups, cap):
    rng = np.random.default_rng(22)
    p, shard, vocab, rows = 2, 512, 1001, 333
    x = make_logits(rng, rows, vocab, "bf16")
    tokens = rng.integers(-1, vocab, rows)
    a = rng.normal(size=rows).astype(np.float32)
    g = groups(p)
    check_log_probs(g, x, p, shard, tokens, "bf16", k=4, cap=cap)
    assert 0 < g.last_launch()["ctas"] <= cap
    check_backward(g, x, p, shard, tokens, "bf16", a, a, cap=cap)
    assert 0 < g.last_launch()["ctas"] <= cap
    ids, t = make_teacher(rng, rows, vocab, 5)
    check_distill(g, x, p, shard, ids, t, "bf16", w=a, cap=cap)
    assert 0 < g.last_launch()["ctas"] <= cap
    # a few rows under a cap, and more rows than the device holds CTAs
    check_log_probs(g, x[:2], p, shard, tokens[:2], "bf16", k=4, cap=cap)
    big = make_logits(rng, 3000, 40, "bf16")
    check_log_probs(g, big, p, 24, rng.integers(0, 40, 3000), "bf16", k=2, cap=cap if cap > 3 else 0)


RING_THREADS = 640  # the persistent kernel of long rows

# ranks, shard, vocab, datatype, cap, rows: clusters of 1, 2, 4, 5 to 8 CTAs, one
# of them or two, and rows enough for every slot and barrier to be used in turn
RING = [(1, 33000, 33000, "bf16", 1, 29), (3, 11000, 32999, "bf16", 2, 61), (2, 24000, 48000, "f32", 4, 9),
        (8, 16384, 131072, "bf16", 8, 23), (5, 20001, 100003, "f32", 8, 13), (2, 50001, 100002, "f32", 7, 11),
        (4, 65536, 262144, "bf16", 8, 5)]


@pytest.mark.parametrize("p,shard,vocab,dtype,cap,rows", RING)
def test_long_rows(groups, p, shard, vocab, dtype, cap, rows):
    """Rows that stay in shared memory between their sum and their gradient.
    Under a cap few rows are enough for that kernel."""
    rng = np.random.default_rng(vocab + rows)
    x = make_logits(rng, rows, vocab, dtype)
    lowest = torch.finfo(TORCH[dtype]).min
    x[1] = float("-inf")
    x[2, 10:] = float("-inf")
    x[3] = lowest
    x[4, : vocab // 2] = lowest
    w = rng.normal(size=rows).astype(np.float32)
    w[0] = 0.0
    g = groups(p)
    for k, temperature, known, kw in ((33, 1.0, False, {}), (128, 0.7, True, dict(gap=3, gap_out=1, offset=1, offset_out=2)),
                                      (2, 2.0, False, dict(in_place=True, gap=1))):
        ids, t = make_teacher(rng, rows, vocab, k)
        ids[-1] = -1                       # no entries
        ids[0, 0], ids[0, -1] = 0, vocab - 1
        if k > 2:
            ids[-2, 1::2] = ids[-2, 0]     # a column named many times
        lse = (rng.normal(size=rows) + 4).astype(np.float32) if known else None
        first = check_distill(g, x, p, shard, ids, t, dtype, temperature, lse, w, "bf16" if known else "f32",
                              cap=cap, ways=("step",), **kw)
        info = g.last_launch()
        # many odd segments have too many edge elements for it
        assert info["ctas"] <= cap and (info["threads"] == RING_THREADS) == (p <= 5 or "offset" not in kw), info
        again = check_distill(g, x, p, shard, ids, t, dtype, temperature, lse, w, "bf16" if known else "f32",
                              cap=cap, ways=("step",), **kw)
        assert torch.equal(first[0][0], again[0][0])
        assert all(torch.equal(m, n) for m, n in zip(first[0][2], again[0][2]))


def test_long_rows_uncapped_and_special(groups):
    """The same kernel over the whole device, with NaN and infinite logits, and
    against the forward and the gradient apart."""
    p, shard, vocab, rows, dtype = 4, 16384, 65536, 800, "bf16"  # enough that it takes them uncapped
    rng = np.random.default_rng(40)
    x = make_logits(rng, rows, vocab, dtype)
    x[5, 9000] = float("nan")
    x[6, 3] = float("inf")
    ids, t = make_teacher(rng, rows, vocab, 8)
    w = np.abs(rng.normal(size=rows)).astype(np.float32) + 0.1
    g = groups(p)
    logits = cut(x, p, shard)
    out = {}
    for way in ("one", "two"):
        loss, st, grads = f32(rows), f32(rows, 2), grad_buffers(x, p, shard, 0, 0)
        if way == "one":
            g.distill(logits, dev(ids, torch.int64), dev(t), loss, st, weights=dev(w), grads=grads)
            assert g.last_launch()["threads"] == RING_THREADS
        else:
            g.distill(logits, dev(ids, torch.int64), dev(t), loss, st)
            g.distill_backward(logits, dev(ids, torch.int64), dev(t), st, dev(w), grads)
        torch.cuda.synchronize()
        assert g.query_error() == tccl.tcclSuccess
        out[way] = host(loss), glue(grads, vocab)[0]
    bad = np.zeros(rows, bool)
    bad[[5, 6]] = True
    for loss, grad in out.values():
        assert np.isnan(loss[bad]).all() and np.isfinite(loss[~bad]).all()
        assert np.isnan(grad[bad]).all() and np.isfinite(grad[~bad]).all()
    keep = ~bad & (np.arange(rows) % 3 != 1)
    loss, tl, grad, tg = distill_bounds(x[torch.from_numpy(keep)], ids[keep], t[keep].astype(np.float32), 1.0, None, w[keep])
    for got_loss, got in out.values():
        close(got_loss[keep], loss, tl, "loss")
        close_grad(got[keep], grad, tg, dtype, "gradient")


def test_long_rows_wait_timeout(groups):
    """A wait of the persistent kernel that runs out is reported, ends the
    kernel, and leaves the next call right."""
    p, shard, vocab, rows = 2, 65536, 131072, 12
    rng = np.random.default_rng(41)
    x = make_logits(rng, rows, vocab, "bf16")
    ids, t = make_teacher(rng, rows, vocab, 4)
    w = rng.normal(size=rows).astype(np.float32)
    g = tccl.Group(p)
    try:
        g.set_config(wait_timeout_ms=30.0)
        logits, grads, loss = cut(x, p, shard), grad_buffers(x, p, shard, 0, 0), f32(rows)
        assert tccl.tcclGroupInjectWaitTimeout(g.handle, True, 2.0) == tccl.tcclSuccess
        g.distill(logits, dev(ids, torch.int64), dev(t), loss, weights=dev(w), grads=grads, cta_cap=8)
        assert g.last_launch()["threads"] == RING_THREADS
        assert g.query_error() == tccl.tcclDeviceTimeout
        assert tccl.tcclGroupInjectWaitTimeout(g.handle, False, 0.0) == tccl.tcclSuccess
        check_distill(g, x, p, shard, ids, t, "bf16", w=w, cap=8, ways=("step",))
        assert g.last_launch()["threads"] == RING_THREADS
    finally:
        g.close()


def test_rows_far_apart(groups):
    """Element offsets past 2^32: the last row starts 4.4e9 elements in."""
    rng = np.random.default_rng(23)
    rows, vocab, stride = 2101, 700, 1 << 21
    x = make_logits(rng, rows, vocab, "bf16")
    raw = torch.empty(rows, stride, dtype=torch.bfloat16, device="cuda")
    raw[:, :vocab] = x.cuda()
    tokens = rng.integers(0, vocab, rows)
    a = rng.normal(size=rows).astype(np.float32)
    g = groups(1)
    check_log_probs(g, x, 1, vocab, tokens, "bf16", k=2, logits=[raw[:, :vocab]])
    grads = [raw[:, 1024:1024 + vocab]]
    g.log_probs_backward([raw[:, :vocab]], dev(tokens, torch.int64), stats_of(x, 1.0), dev(a), grads)
    lp, _, _ = vo.log_softmax(x.double().numpy(), 1.0)
    exp = vo.log_probs_backward(x.double().numpy(), tokens, 1.0, a, None)
    tol = np.abs(a)[:, None] * (np.exp(lp) * (tol_p(lp, vocab) + 8 * U) + 4 * U)
    check_grads(grads, exp, tol, "bf16", vocab, "grads")
    ids, t = make_teacher(rng, rows, vocab, 3)
    loss, tl, eg, tg = distill_bounds(x, ids, t.astype(np.float32), 1.0, None, a)
    got = f32(rows)
    g.distill([raw[:, :vocab]], dev(ids, torch.int64), dev(t), got, weights=dev(a), grads=grads)
    close(host(got), loss, tl, "loss")
    check_grads(grads, eg, tg, "bf16", vocab, "grads")
    del raw, grads
    torch.cuda.empty_cache()


def test_streams_graphs_and_repeats(groups):
    """Another stream, a captured graph replayed on new data in the same
    buffers, and the same bits from the same call."""
    rng = np.random.default_rng(24)
    p, shard, vocab, rows, k = 4, 1024, 4000, 6, 10
    g = groups(p)
    x = make_logits(rng, rows, vocab, "bf16")
    logits = cut(x, p, shard)
    tokens = dev(rng.integers(0, vocab, rows), torch.int64)
    ids, t = make_teacher(rng, rows, vocab, k)
    ids, t, w = dev(ids, torch.int64), dev(t), dev(rng.normal(size=rows))

    def buffers():
        return dict(lp=f32(rows), ent=f32(rows), st=f32(rows, 2), top=f32(rows, k),
                    tid=torch.zeros(rows, k, dtype=torch.int64, device="cuda"), loss=f32(rows),
                    g1=[torch.zeros_like(m) for m in logits], g2=[torch.zeros_like(m) for m in logits])

    def step(o):
        g.log_probs(logits, tokens, o["lp"], o["ent"], o["st"], o["top"], o["tid"], vocab=vocab)
        g.log_probs_backward(logits, tokens, o["st"], w, o["g1"], entropy=o["ent"], d_entropy=w, vocab=vocab)
        g.distill(logits, ids, t, o["loss"], weights=w, grads=o["g2"], vocab=vocab)

    def same(a, b):
        for key in a:
            for u, v in zip(*((m if isinstance(m, list) else [m]) for m in (a[key], b[key]))):
                assert torch.equal(u, v), key

    one, two, three = buffers(), buffers(), buffers()
    step(one)
    step(two)
    torch.cuda.synchronize()
    same(one, two)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(three)
    for m in logits:
        m.mul_(0.5)
    graph.replay()
    step(two)
    torch.cuda.synchronize()
    same(two, three)


def test_refusals(groups):
    g = groups(2)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    L, G = [bf(4, 64), bf(4, 64)], [bf(4, 64), bf(4, 64)]
    tok, st = torch.zeros(4, dtype=torch.int64, device="cuda"), f32(4, 2)
    lp, w = f32(4), f32(4)
    ids, t = torch.zeros(4, 3, dtype=torch.int64, device="cuda"), f32(4, 3)
    bad, ok = tccl.tcclInvalidArgument, tccl.tcclSuccess

    def shape(**kw):
        d = dict(rows=4, vocab=128, shard=64, row_stride=64, datatype=1, temperature=1.0)
        d.update(kw)
        return tccl.tcclVocab_t(**d)

    def fwd(s, L=L, tok=tok, lp=lp, **kw):
        return tccl.tcclLogProbs(g.handle, L, s, tok, lp, **kw)

    assert fwd(shape()) == ok
    for kw in (dict(vocab=0), dict(vocab=129), dict(shard=0), dict(row_stride=63), dict(datatype=2),
               dict(datatype=7), dict(temperature=0.0), dict(temperature=-1.0),
               dict(temperature=float("nan")), dict(temperature=float("inf")), dict(temperature=1e-6),
               dict(rows=1 << 31), dict(shard=1 << 30), dict(row_stride=1 << 31)):
        assert fwd(shape(**kw)) == bad, kw
    assert fwd(shape(rows=0)) == ok
    assert fwd(shape(), L=[L[0], 0]) == bad
    assert fwd(shape(), L=[L[0], L[1].data_ptr() + 1]) == bad
    assert fwd(shape(), tok=tok.data_ptr() + 4) == bad
    assert fwd(shape(), tok=None) == bad and fwd(shape(), lp=None) == bad
    assert fwd(shape(), tok=None, lp=None, stats=st) == ok
    assert fwd(shape(), top_k=3) == bad
    assert fwd(shape(), top_k=3, top_log_probs=t, top_ids=ids) == ok
    assert fwd(shape(), top_k=-1, top_log_probs=t, top_ids=ids) == bad
    assert fwd(shape(), top_k=129, top_log_probs=f32(4, 129), top_ids=ids) == bad
    assert fwd(shape(), entropy=lp) == bad  # two outputs in one place
    assert fwd(shape(), lp=L[1]) == bad     # an output over an input
    null = tccl.ctypes.c_void_p()
    assert tccl.tcclLogProbs(null, L, shape(), tok, lp) == bad

    def bwd(s, G=G, stride=64, tok=tok, st=st, da=w, ent=None, de=None):
        return tccl.tcclLogProbsBackward(g.handle, L, s, tok, st, ent, da, de, G, stride)

    assert bwd(shape()) == ok and bwd(shape(), G=L) == ok
    assert bwd(shape(), stride=63) == bad
    assert bwd(shape(), G=[L[1], L[0]]) == bad          # each other's logits
    assert bwd(shape(), G=[G[0], G[0]]) == bad
    assert bwd(shape(), G=[G[0].data_ptr() + 64, G[1]], stride=128) == bad
    assert bwd(shape(), tok=None) == bad and bwd(shape(), st=None) == bad and bwd(shape(), da=None) == bad
    assert bwd(shape(), de=w) == bad                    # entropy's gradient without the entropy
    assert bwd(shape(), de=w, ent=lp) == ok
    assert bwd(shape(), st=G[0]) == bad
    assert bwd(shape(rows=2, row_stride=128), G=L, stride=64) == bad  # in place, another stride

    def dis(s, k=3, ids=ids, t=t, td=0, loss=lp, **kw):
        return tccl.tcclDistill(g.handle, L, s, ids, t, td, None, k, loss, **kw)

    assert dis(shape()) == ok and dis(shape(), weights=w, grads=G, grad_stride=64) == ok
    assert dis(shape(), k=0) == bad and dis(shape(), k=129) == bad
    assert dis(shape(), td=2) == bad and dis(shape(), ids=None) == bad and dis(shape(), t=None) == bad
    assert dis(shape(), loss=None) == bad
    assert dis(shape(), weights=w) == bad and dis(shape(), grads=G, grad_stride=64) == bad
    assert dis(shape(), weights=w, grads=G, grad_stride=32) == bad
    assert dis(shape(), weights=lp, grads=G, grad_stride=64) == bad
    assert tccl.tcclDistillBackward(g.handle, L, shape(), ids, t, 0, None, 3, None, w, G, 64) == bad
    assert tccl.tcclDistillBackward(g.handle, L, shape(), ids, t, 0, None, 3, st, w, G, 64) == ok
    torch.cuda.synchronize()

    # the Group methods check what the C call cannot see
    for call in (lambda: g.log_probs(L[:1], tok, lp), lambda: g.log_probs([L[0], bf(4, 32)], tok, lp),
                 lambda: g.log_probs(L, tok[:3], lp), lambda: g.log_probs(L, tok.int(), lp),
                 lambda: g.log_probs(L, tok, lp, top_ids=ids), lambda: g.log_probs(L, tok, lp, vocab=0),
                 lambda: g.log_probs([m.t() for m in L], tok, lp),
                 lambda: g.log_probs([m.half() for m in L], tok, lp),
                 lambda: g.log_probs([m.cpu() for m in L], tok, lp),
                 lambda: g.log_probs_backward(L, tok, st, w, [bf(4, 64), bf(3, 64)]),
                 lambda: g.log_probs_backward(L, tok, st, w, [f32(4, 64), f32(4, 64)]),
                 lambda: g.log_probs_backward(L, tok, f32(4), w, G),
                 lambda: g.distill(L, ids, t[:, :2].contiguous(), lp), lambda: g.distill(L, ids, t, f32(3)),
                 lambda: g.distill(L, ids, t, lp, weights=w),
                 lambda: g.distill_backward(L, ids, t, st, f32(3), G)):
        with pytest.raises(tccl.TcclError) as e:
            call()
        assert e.value.code == bad
    empty = [bf(0, 64), bf(0, 64)]
    g.log_probs(empty, tok[:0], lp[:0])
    g.distill(empty, ids[:0], t[:0], lp[:0], weights=w[:0], grads=[bf(0, 64), bf(0, 64)])
