"""Cases for the vocabulary-parallel operators: log probabilities of given
tokens (with entropy and the top alternatives) and distillation from a
teacher's top logits, forward and backward, over logits that P ranks hold cut
by columns.

Rank r holds columns [r * shard, (r + 1) * shard) of every row; columns at or
past `vocab` are padding. With z = x / temperature over the valid columns and
lse = log(sum_j exp(z_j)):

  log_probs   z[token] - lse, the entropy -sum_j p_j log p_j, and the top_k
              largest columns (equal values: the lower column first) with their
              log probabilities; a column at -inf is never listed (id -1, -inf).
              A row whose every column is -inf has log probability -inf,
              entropy 0. A row with token -1 is not scored: all zeros, no
              alternatives.
  log_probs_backward
              (a [j == token] - p_j (a + b (log p_j + entropy))) / temperature
              with a, b the gradients of log probability and entropy.
  distill     sum_k q_k (log q_k - log p[id_k]), q the teacher's softmax over
              its K kept logits (or exp(t / temperature - teacher_lse) where the
              log-sum of its whole row is given); entries with id -1 are empty.
              With weights w also the gradient w (Q p_j - q_j) / temperature,
              Q = sum_k q_k, q_j = 0 where the teacher kept nothing.
  distill_backward
              that gradient alone, from the forward's row statistics.

`own = False` computes them in elementary torch operations in 32 bits,
rounded once at the end; `own = True` calls this package.
"""
import math

import torch

own = False

NEG = float("-inf")
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def _case(op, rows, vocab, ranks, dtype="bf16", **kw):
    """op: log_probs, log_probs_backward, distill (loss only), distill_step
    (loss and gradient in one call) or distill_backward. align: a rank's
    columns are a multiple of it (the last rank's rest is padding). gap: unused
    elements between rows. unscored: share of rows without a token (or with
    weight 0). banned: share of columns at -inf."""
    case = {"op": op, "rows": rows, "vocab": vocab, "ranks": ranks, "dtype": dtype, "align": 1,
            "gap": 0, "temperature": 1.0, "top_k": 0, "entropy": op.startswith("log_probs"),
            "unscored": 0.0, "banned": 0.0, "teacher_k": 0, "teacher_dtype": "f32",
            "teacher_lse": False}
    case.update(kw)
    return case


def listed():
    out = []

    def add(name, *a, **kw):
        out.append({"name": name, **_case(*a, **kw)})

    # one decoded token with the 20 alternatives a serving interface may return
    add("logprobs_decode_1", "log_probs", 1, 131072, 8, align=64, top_k=20)
    # a decode batch
    add("logprobs_decode_64", "log_probs", 64, 131072, 8, align=64, top_k=5)
    # scoring rollouts before a policy update: no alternatives, prompt rows unscored
    add("logprobs_score_4096", "log_probs", 4096, 131072, 8, align=64, unscored=0.125)
    # a teacher writing the top logits that a student is distilled from
    add("logprobs_teacher_1024", "log_probs", 1024, 131072, 4, align=64, top_k=64, entropy=False)
    # sampling under a grammar's mask, fp32 logits, an odd vocabulary over three ranks
    add("logprobs_masked_f32_777", "log_probs", 777, 50021, 3, "f32", top_k=8, temperature=0.7,
        banned=0.5)
    # a policy update's gradient with an entropy bonus
    add("logprobs_grad_4096", "log_probs_backward", 4096, 131072, 8, align=64, unscored=0.25)
    # a small fine-tuning batch: cross entropy's gradient, odd sizes, fp32
    add("logprobs_grad_f32_37", "log_probs_backward", 37, 32003, 2, "f32", entropy=False)
    # evaluating a student: a few rows, and a whole batch
    add("distill_eval_8", "distill", 8, 32768, 2, align=64, teacher_k=16)
    add("distill_eval_2048", "distill", 2048, 131072, 8, align=64, teacher_k=64, temperature=2.0)
    # a distillation step: loss and gradient together
    add("distill_step_4096", "distill_step", 4096, 131072, 8, align=64, teacher_k=64,
        temperature=2.0, unscored=0.125)
    # the same on fp32 logits of an odd vocabulary over five ranks, teacher's whole-row sum known
    add("distill_step_f32_301", "distill_step", 301, 100003, 5, "f32", teacher_k=33,
        teacher_lse=True)
    # the gradient apart from the loss (a weight known only afterwards), the widest vocabulary
    add("distill_grad_1024", "distill_backward", 1024, 262144, 4, align=64, teacher_k=128,
        teacher_dtype="bf16", unscored=0.25)
    return out


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["log_probs", "log_probs", "log_probs_backward", "distill", "distill_step",
                     "distill_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    vocab = _log_int(rng, 1000, 262144)
    limit = (1 << 29) // (vocab * BYTES[dtype] // 2)
    rows = min(_log_int(rng, 1, 4096), max(1, limit))
    kw = {"align": rng.choice([1, 8, 64, 128]), "gap": rng.choice([0, 0, 8, 3]),
          "temperature": rng.choice([1.0, 1.0, 0.6, 2.0]),
          "unscored": rng.choice([0.0, 0.25])}
    if op == "log_probs":
        kw["top_k"] = rng.choice([0, 1, 5, 20, 64])
        kw["banned"] = rng.choice([0.0, 0.0, 0.9])
    if op.startswith("log_probs"):
        kw["entropy"] = rng.random() < 0.7
    else:
        kw["teacher_k"] = rng.choice([1, 7, 32, 64, 128])
        kw["teacher_dtype"] = rng.choice(["f32", "bf16"])
        kw["teacher_lse"] = rng.random() < 0.3
    return _case(op, rows, vocab, rng.choice([1, 2, 3, 4, 8, 16]), dtype, **kw)


def _shard(case):
    per = -(-case["vocab"] // case["ranks"])
    return -(-per // case["align"]) * case["align"]


def _inputs(case, seed):
    """Everything a caller holds: the logits per rank, and the tokens or the
    teacher's entries, with row statistics where only the gradient is asked."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, vocab, ranks = case["rows"], case["vocab"], case["ranks"]
    dtype, shard, op = TORCH[case["dtype"]], _shard(case), case["op"]

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    def uniform(*shape):
        return torch.rand(*shape, device=dev, generator=gen)

    # a column bias shared by all rows, a row offset, noise; the top of a row
    # is as sharp as a trained model's (its largest probability mostly 0.1-0.9)
    x = normal(rows, vocab).mul_(1.5).add_(normal(vocab).mul_(1.5)).add_(normal(rows, 1).mul_(2.0))
    peak = torch.randint(0, vocab, (rows, 4), device=dev, generator=gen)
    x.scatter_add_(1, peak, uniform(rows, 4) * 12.0)
    x = x.to(dtype)
    if case["banned"]:
        keep = uniform(rows, vocab) >= case["banned"]
        if rows > 2:
            keep[1] = False            # a mask that leaves nothing
            keep[2] = False
            keep[2, [3, vocab // 2]] = True  # ... and one that leaves two columns
        x.masked_fill_(~keep, NEG)
    # a permutation, so that exactly that share of the rows is unscored
    unscored = torch.randperm(rows, device=dev, generator=gen)[:int(rows * case["unscored"])]
    s = {"temperature": case["temperature"], "vocab": vocab}
    if op.startswith("log_probs"):
        best = x.float().argmax(1)
        other = torch.randint(0, vocab, (rows,), device=dev, generator=gen)
        s["tokens"] = torch.where(uniform(rows) < 0.7, best, other)
        s["tokens"][unscored] = -1
        s["top_k"], s["entropy"] = case["top_k"], case["entropy"]
        if op == "log_probs_backward":
            s["d_log_probs"] = normal(rows) / rows
            s["d_entropy"] = torch.full((rows,), 0.01 / rows, device=dev) if case["entropy"] else None
    else:
        y = x.float() * 0.9 + normal(rows, vocab)
        top, ids = y.topk(case["teacher_k"], 1)
        s["teacher_logits"] = top.to(TORCH[case["teacher_dtype"]])
        ids[uniform(rows, case["teacher_k"]) < 0.02] = -1  # a few empty entries
        s["teacher_ids"] = ids
        s["teacher_lse"] = (torch.logsumexp(y / case["temperature"], 1)
                            if case["teacher_lse"] else None)
        del y
        if op != "distill":
            s["weights"] = torch.full((rows,), 1.0 / rows, device=dev)
            s["weights"][unscored] = 0.0
    if op.endswith("_backward"):
        z = x.float() / case["temperature"]
        top = z.max(1).values
        s["stats"] = torch.stack([x.float().max(1).values, (z - top[:, None]).exp().sum(1).log()], 1)
        p = torch.softmax(z, 1)
        s["entropy_value"] = -(p * torch.log(p.clamp_min(1e-38))).sum(1) if case.get("entropy") else None
        del z, p
    s["logits"] = []
    for r in range(ranks):
        part = x[:, min(r * shard, vocab):min((r + 1) * shard, vocab)]
        whole = torch.zeros(rows, shard + case["gap"], device=dev, dtype=dtype)
        whole[:, :part.shape[1]] = part
        s["logits"].append(whole[:, :shard])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["op"] = case["op"]
    if not own:
        return s
    import collective_communication_planner_gb300 as tccl

    rows, dev = case["rows"], s["logits"][0].device
    g = s["group"] = tccl.Group(case["ranks"])
    kw = {"vocab": s["vocab"], "temperature": s["temperature"]}

    def out(*shape, dtype=torch.float32):
        return torch.empty(*shape, device=dev, dtype=dtype)

    if s["op"] == "log_probs":
        k = s["top_k"]
        s["out"] = [out(rows), out(rows) if s["entropy"] else None, out(rows, k) if k else None,
                    out(rows, k, dtype=torch.int64) if k else None]
        lp, ent, top, ids = s["out"]
        s["call"] = g.prepare_log_probs(s["logits"], s["tokens"], lp, entropy=ent,
                                        top_log_probs=top, top_ids=ids, **kw)
        return s
    grads = [out(rows, t.shape[1], dtype=t.dtype) for t in s["logits"]]
    if s["op"] == "log_probs_backward":
        s["out"] = [grads]
        s["call"] = g.prepare_log_probs_backward(
            s["logits"], s["tokens"], s["stats"], s["d_log_probs"], grads,
            entropy=s["entropy_value"], d_entropy=s["d_entropy"], **kw)
        return s
    teacher = (s["teacher_ids"], s["teacher_logits"])
    kw["teacher_lse"] = s["teacher_lse"]
    if s["op"] == "distill_backward":
        s["out"] = [grads]
        s["call"] = g.prepare_distill_backward(s["logits"], *teacher, s["stats"], s["weights"],
                                               grads, **kw)
        return s
    s["out"] = [out(rows)]
    if s["op"] == "distill_step":
        s["out"].append(grads)
        kw.update(weights=s["weights"], grads=grads)
    s["call"] = g.prepare_distill(s["logits"], *teacher, s["out"][0], **kw)
    return s


def _cut(grad, s):
    """The [rows, vocab] gradient as the ranks hold it, padding columns zero."""
    shard, vocab = s["logits"][0].shape[1], s["vocab"]
    out = []
    for r, x in enumerate(s["logits"]):
        part = grad[:, min(r * shard, vocab):min((r + 1) * shard, vocab)].to(x.dtype)
        whole = torch.zeros(x.shape, device=x.device, dtype=x.dtype)
        whole[:, :part.shape[1]] = part
        out.append(whole)
    return out


def _plain_top(x, logp, k):
    """Column order: value down, then column up, as one 64-bit key."""
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64) << 32
    key -= torch.arange(x.shape[1], device=x.device)
    ids = key.topk(min(k, x.shape[1]), 1).indices
    if ids.shape[1] < k:
        ids = torch.cat([ids, ids[:, :1].expand(-1, k - ids.shape[1])], 1)
    val = logp.gather(1, ids)
    none = x.gather(1, ids) == NEG
    return torch.where(none, NEG, val), torch.where(none, -1, ids)


def _plain(s):
    op, t = s["op"], s["temperature"]
    x = torch.cat([l.float() for l in s["logits"]], 1)[:, :s["vocab"]]
    z = x / t
    if op.endswith("_backward"):
        logp = z - (s["stats"][:, :1] / t + s["stats"][:, 1:])
    else:
        top = z.max(1, keepdim=True).values
        top = torch.where(top == NEG, 0.0, top)
        logp = (z - top) - (z - top).exp().sum(1, keepdim=True).log()
        logp = torch.where(x == NEG, NEG, logp)
    if op.startswith("log_probs"):
        on = s["tokens"] >= 0
        token = s["tokens"].clamp_min(0)[:, None]
        if op == "log_probs":
            res = [torch.where(on, logp.gather(1, token)[:, 0], 0.0), None, None, None]
            if s["entropy"]:
                h = -torch.where(logp == NEG, 0.0, logp.exp() * logp).sum(1)
                res[1] = torch.where(on, h, 0.0)
            if s["top_k"]:
                val, ids = _plain_top(x, logp, s["top_k"])
                res[2] = torch.where(on[:, None], val, NEG)
                res[3] = torch.where(on[:, None], ids, -1)
            return res
        a = s["d_log_probs"][:, None]
        p = logp.exp()
        if s["d_entropy"] is None:
            g = p * -a
        else:
            inner = torch.where(p == 0, 0.0, logp + s["entropy_value"][:, None])
            g = -p * (a + s["d_entropy"][:, None] * inner)
        g.scatter_add_(1, token, a)
        return [_cut(torch.where(on[:, None], g / t, 0.0), s)]
    has = s["teacher_ids"] >= 0
    ids = s["teacher_ids"].clamp_min(0)
    tz = torch.where(has, s["teacher_logits"].float() / t, NEG)
    if s["teacher_lse"] is None:
        top = tz.max(1, keepdim=True).values
        top = torch.where(top == NEG, 0.0, top)
        logq = (tz - top) - (tz - top).exp().sum(1, keepdim=True).log()
    else:
        logq = tz - s["teacher_lse"][:, None]
    q = torch.where(has, logq.exp(), 0.0)
    res = []
    if op != "distill_backward":
        res.append(torch.where(q > 0, q * (logq - logp.gather(1, ids)), 0.0).sum(1))
    if op != "distill":
        g = logp.exp() * q.sum(1, keepdim=True)
        g.scatter_add_(1, ids, -q)
        w = s["weights"][:, None] / t
        res.append(_cut(torch.where(w == 0, 0.0, g * w), s))
    return res


def run(state):
    if own:
        state["call"]()
        return state["out"]
    return _plain(state)


def exact(case, seed):
    """The definitions in 64 bits, a block of rows at a time."""
    s = _inputs(case, seed)
    op, vocab, t = case["op"], case["vocab"], case["temperature"]
    rows, shard = case["rows"], _shard(case)
    dev = s["logits"][0].device
    f64 = torch.float64
    step = max(1, (1 << 26) // vocab)
    loss, ent, tops, ids_out = [], [], [], []
    grads = [torch.zeros(rows, shard, dtype=f64, device=dev) for _ in range(case["ranks"])]

    def put(lo, g):
        for r, whole in enumerate(grads):
            a, b = min(r * shard, vocab), min((r + 1) * shard, vocab)
            whole[lo:lo + g.shape[0], :b - a] = g[:, a:b]

    for lo in range(0, rows, step):
        hi = min(rows, lo + step)
        raw = torch.cat([l[lo:hi] for l in s["logits"]], 1)[:, :vocab].to(f64)
        n = hi - lo
        lp = raw / t - torch.logsumexp(raw / t, 1, keepdim=True)
        empty = torch.isneginf(raw).all(1)
        lp[empty] = NEG
        prob = lp.exp()
        if op.startswith("log_probs"):
            tok = s["tokens"][lo:hi]
            off = tok < 0
            at = torch.where(off, 0, tok)
            h = -torch.special.xlogy(prob, prob).sum(1)
            if op == "log_probs":
                got = lp[torch.arange(n, device=dev), at]
                got[off] = 0.0
                h[off] = 0.0
                loss.append(got)
                ent.append(h)
                if case["top_k"]:
                    v = torch.full((n, case["top_k"]), NEG, dtype=f64, device=dev)
                    i = torch.full((n, case["top_k"]), -1, dtype=torch.int64, device=dev)
                    k = min(case["top_k"], vocab)
                    # a stable sort keeps the lower column first among equals
                    order = torch.sort(-raw, dim=1, stable=True).indices[:, :k]
                    v[:, :k] = lp.gather(1, order)
                    i[:, :k] = order
                    i[torch.isneginf(v)] = -1
                    v[off], i[off] = NEG, -1
                    tops.append(v)
                    ids_out.append(i)
                continue
            a = s["d_log_probs"][lo:hi].to(f64)[:, None]
            hot = torch.zeros_like(prob)
            hot[torch.arange(n, device=dev), at] = 1.0
            g = a * (hot - prob)
            if case["entropy"]:
                b = s["d_entropy"][lo:hi].to(f64)[:, None]
                g -= b * (torch.special.xlogy(prob, prob) + prob * h[:, None])
            g[off] = 0.0
            put(lo, g / t)
            continue
        has = s["teacher_ids"][lo:hi] >= 0
        ids = torch.where(has, s["teacher_ids"][lo:hi], 0)
        tz = s["teacher_logits"][lo:hi].to(f64) / t
        tz[~has] = NEG
        if s["teacher_lse"] is None:
            q = torch.softmax(tz, 1)
            q[~has.any(1)] = 0.0
        else:
            q = (tz - s["teacher_lse"][lo:hi].to(f64)[:, None]).exp()
        picked = lp.gather(1, ids)
        cross = torch.where(q > 0, q * picked, 0.0)
        loss.append((torch.special.xlogy(q, q) - cross).sum(1))
        if op != "distill":
            g = prob * q.sum(1, keepdim=True)
            g.scatter_add_(1, ids, -q)
            put(lo, g * (s["weights"][lo:hi].to(f64)[:, None] / t))
    if op == "log_probs":
        k = case["top_k"]
        return [torch.cat(loss), torch.cat(ent) if case["entropy"] else None,
                torch.cat(tops) if k else None, torch.cat(ids_out) if k else None]
    if op.endswith("_backward"):
        return [grads]
    return [torch.cat(loss)] + ([grads] if op == "distill_step" else [])


def work(case):
    """Logits of the scored rows read once, gradients of all rows written once
    (padding columns among them), the row vectors; operations: one exponential
    and about four additions or products an element in a forward pass, six in a
    gradient."""
    rows, vocab, es, op = case["rows"], case["vocab"], BYTES[case["dtype"]], case["op"]
    skipped = int(rows * case["unscored"])
    if op in ("distill", "distill_step"):
        skipped = 0  # the loss of a row with weight 0 is still computed
    read = (rows - skipped) * vocab
    row_bytes, flops = 0, 0
    if op.startswith("log_probs"):
        row_bytes = 8 + 4 + 4 * case["entropy"] + 12 * case["top_k"]
        if op.endswith("_backward"):
            row_bytes = 8 + 8 + 4 + 8 * case["entropy"]
    else:
        row_bytes = case["teacher_k"] * (8 + BYTES[case["teacher_dtype"]]) + 4 * case["teacher_lse"] + 4
        if op != "distill":
            row_bytes += 4
        if op == "distill_backward":
            row_bytes += 4
    total = read * es + rows * row_bytes
    if not op.endswith("_backward"):
        flops += 5 * read
    if op in ("log_probs_backward", "distill_backward", "distill_step"):
        total += rows * case["ranks"] * _shard(case) * es
        flops += 6 * read
    return {"bytes": total, "flops": flops}
