"""Cases of the windowed causal attention, its learned relative position bias and
the top-logit distillation loss, for timing and for checking.

Attention (op "attention"), per sequence, head width 64, scale 1/8:
  query i sees key j when j <= i and (i - j < window or j < sinks), within the
  sequence's length; scores s_ij = q_i . k_j / 8 + table[bucket(i - j), head];
  o_i = sum_j softmax_j(s_ij) v_j, lse_i = log sum_j e^{s_ij}.  A padded row
  (i >= length) has o = 0, lse = -inf and zero gradients.
Distillation (op "distill"), per row of student logits z and a teacher's top
logits t_k at tokens idx_k, p = softmax(t / T) over the slots with idx_k >= 0:
  loss = kd T^2 sum_k p_k (log p_k - log softmax(z / T)[idx_k])
       + ce (lse(z) - z[next token]),
  dz   = kd T (softmax(z / T) - sum_k p_k onehot(idx_k))
       + ce (softmax(z) - onehot(next token)).
"""
import math

import torch

own = False  # true: run() calls the library; false: plain torch

HD = 64


def _attention(name, nseq, seq, heads, kv_heads, window, sinks, buckets, max_distance, fill, train):
    return {"name": name, "op": "attention", "nseq": nseq, "seq": seq, "heads": heads, "kv_heads": kv_heads,
            "window": window, "sinks": sinks, "buckets": buckets, "max_distance": max_distance, "fill": fill,
            "train": train}


def _distill(name, rows, vocab, pad, topk, dtype, temperature, kd, ce, seq, train):
    return {"name": name, "op": "distill", "rows": rows, "vocab": vocab, "pad": pad, "topk": topk, "dtype": dtype,
            "temperature": temperature, "kd": kd, "ce": ce, "seq": seq, "train": train}


def listed():
    return [
        # a few short prompts: one tile per head, launch latency counts
        _attention("attention_small_train", 3, 19, 4, 2, 8, 2, 8, 16, 1.0, True),
        # one micro-batch of the memory-scaling workload (4 x 512 tokens, 16 heads), local layers
        _attention("attention_window_fwd", 4, 512, 16, 16, 128, 4, 0, 0, 1.0, False),
        _attention("attention_window_train", 4, 512, 16, 16, 128, 4, 0, 0, 1.0, True),
        # the same micro-batch, every earlier token visible, positions by a learned table
        _attention("attention_bias_train", 4, 512, 16, 16, 512, 0, 32, 128, 1.0, True),
        # a padded batch of unequal documents with grouped key/value heads
        _attention("attention_ragged_train", 8, 1000, 12, 4, 300, 3, 32, 200, 0.25, True),
        # a long document read once (evaluation), local layers, grouped heads
        _attention("attention_long_fwd", 1, 16384, 8, 2, 1024, 4, 0, 0, 1.0, False),
        # long-context training, local layers with positions
        _attention("attention_long_train", 1, 8192, 16, 16, 2048, 16, 32, 1024, 1.0, True),
        # long-context training, global layers with positions: the most work
        _attention("attention_full_train", 2, 4096, 16, 16, 4096, 0, 32, 128, 1.0, True),
        # a handful of rows over a toy vocabulary
        _distill("distill_small", 5, 517, 3, 8, "f32", 2.0, 0.5, 0.5, 5, True),
        # a micro-batch of the memory-scaling workload (2048 tokens, vocabulary 32000)
        _distill("distill_train", 2048, 32000, 0, 64, "f32", 2.0, 0.7, 0.3, 512, True),
        # evaluation of few rows over a vocabulary of odd size
        _distill("distill_eval", 100, 50001, 7, 100, "f32", 1.0, 1.0, 0.0, 100, False),
        # a large vocabulary with 16-bit logits
        _distill("distill_large_vocab", 4096, 131072, 0, 32, "bf16", 1.5, 1.0, 0.0, 2048, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    train = rng.random() < 0.7
    if rng.random() < 0.65:
        kv = rng.choice((1, 2, 3, 4, 8))
        heads = kv * rng.choice((1, 1, 2, 3, 4, 8))
        heads, kv = (heads, kv) if heads <= 16 else (16, 8)
        seq = _log_int(rng, 1, 8192)
        most = max(1, min(64, 16 * 2 * 4096 * 4096 // (heads * seq * seq)))
        buckets = rng.choice((0, 2, 8, 17, 32, 32, 64))
        return _attention("", _log_int(rng, 1, most), seq, heads, kv, _log_int(rng, 1, seq),
                          rng.choice((0, 0, 1, 4, 16, 33, 64)), buckets,
                          _log_int(rng, buckets // 2 + 1, 4096) if buckets else 0, rng.choice((1.0, 0.0, 0.5)),
                          train)
    vocab = _log_int(rng, 32, 131072)
    rows = _log_int(rng, 1, min(8192, 4096 * 131072 // (2 * vocab)))
    return _distill("", rows, vocab, rng.choice((0, 0, 8, 5)), _log_int(rng, 1, min(256, vocab)),
                    rng.choice(("f32", "bf16")), rng.uniform(0.5, 4.0), rng.uniform(0.1, 1.0),
                    rng.choice((0.0, 0.5)), _log_int(rng, 1, rows), train)


def _lengths(case):
    """Lengths of the padded batch: from seq down to fill * seq in equal steps."""
    n, s, f = case["nseq"], case["seq"], case["fill"]
    return [s - int((1.0 - f) * s * b) // max(1, n - 1) for b in range(n)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    if case["op"] == "attention":
        rows, h, kv = case["nseq"] * case["seq"], case["heads"], case["kv_heads"]
        st["qkv"] = randn(rows, (h + 2 * kv) * HD).bfloat16()
        st["dout"] = randn(rows, h * HD).bfloat16() if case["train"] else None
        st["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["fill"] < 1.0 else None
        if case["buckets"]:
            # nearer tokens weigh more, each head with a spread of its own
            b = torch.arange(case["buckets"], device="cuda", dtype=torch.float32)[:, None]
            st["table"] = randn(case["buckets"], h) * 0.5 - 2.0 * b / case["buckets"]
        else:
            st["table"] = None
        return st
    rows, vocab, ld = case["rows"], case["vocab"], case["vocab"] + case["pad"]
    z = randn(rows, ld) * 2.0
    teacher = z[:, :vocab] + randn(rows, vocab)
    top = torch.topk(teacher, case["topk"], dim=1)
    st["top_logit"], st["top_idx"] = top.values.contiguous(), top.indices.to(torch.int32).contiguous()
    st["top_idx"][::5, case["topk"] // 2 + 1:] = -1  # rows for which the teacher kept fewer
    st["top_idx"][7::11] = -1                        # and rows that it did not score
    del teacher, top
    st["logits"] = z if case["dtype"] == "f32" else z.bfloat16()
    st["tokens"] = torch.randint(0, vocab, (rows + 1,), generator=g, device="cuda", dtype=torch.int32)
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _bucket_of_distance(n, buckets, max_distance, device):
    """bucket(d) for d = 0..n-1: d itself below buckets // 2, then equal steps of log d up to max_distance."""
    d = torch.arange(n, device=device, dtype=torch.float64)
    me = buckets // 2
    far = torch.log(torch.clamp(d, min=1.0) / me) / math.log(max_distance / me) * (buckets - me)
    far = me + torch.floor(far + 1e-11).clamp(max=buckets - 1 - me)
    return torch.where(d < me, d, far).long()


def _visible(case, lens, device):
    s = case["seq"]
    i = torch.arange(s, device=device)[:, None]
    j = torch.arange(s, device=device)[None, :]
    see = (j <= i) & ((i - j < case["window"]) | (j < case["sinks"]))
    if lens is None:
        return see[None, None]
    n = lens.long()[:, None, None]
    return (see[None] & (i[None] < n) & (j[None] < n))[:, None]


def _plain_attention(st):
    c = st["case"]
    n, s, h, kv = c["nseq"], c["seq"], c["heads"], c["kv_heads"]
    grp = h // kv
    x = st["qkv"].float().view(n, s, h + 2 * kv, HD).transpose(1, 2)
    q, k, v = x[:, :h], x[:, h:h + kv], x[:, h + kv:]
    k, v = k.repeat_interleave(grp, 1), v.repeat_interleave(grp, 1)
    a = torch.matmul(q, k.transpose(2, 3)).mul_(0.125)
    if st["table"] is not None:
        at = torch.arange(s, device=a.device)
        of = _bucket_of_distance(s, c["buckets"], c["max_distance"], a.device)
        a += st["table"].t()[:, of][:, (at[:, None] - at[None, :]).clamp_(min=0)]
    a.masked_fill_(~_visible(c, st["lens"], a.device), float("-inf"))
    m = a.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = a.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(p, v)
    lse = (m + total.log()).squeeze(-1).transpose(1, 2).reshape(n * s, h).contiguous()
    out = {"o": o.transpose(1, 2).reshape(n * s, h * HD).bfloat16(), "lse": lse}
    if not c["train"]:
        return out
    do = st["dout"].float().view(n, s, h, HD).transpose(1, 2)
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds -= (p * ds).sum(-1, keepdim=True)
    ds *= p
    del p
    dq = torch.matmul(ds, k).mul_(0.125)
    dk = torch.matmul(ds.transpose(2, 3), q).mul_(0.125)
    dk, dv = (t.view(n, kv, grp, s, HD).sum(2) for t in (dk, dv))
    out["dqkv"] = torch.cat((dq, dk, dv), 1).transpose(1, 2).reshape(n * s, (h + 2 * kv) * HD).bfloat16()
    if st["table"] is not None:
        # sums over each diagonal i - j = d, then over the distances of each bucket
        wide = torch.zeros(h, 2 * s, s, device=ds.device)
        wide[:, :s] = ds.sum(0)
        by_distance = wide.as_strided((h, s, s), (2 * s * s, s, s + 1)).sum(-1, dtype=torch.float64)
        of = _bucket_of_distance(s, c["buckets"], c["max_distance"], ds.device)
        onehot = (of[:, None] == torch.arange(c["buckets"], device=ds.device)).double()
        out["dtable"] = torch.matmul(by_distance, onehot).t().contiguous().float()
    return out


def _plain_distill(st):
    c = st["case"]
    z = st["logits"][:, :c["vocab"]].float()
    t, idx = st["top_logit"] / c["temperature"], st["top_idx"].long()
    kept = idx >= 0
    some = kept.any(1, keepdim=True)
    t = t.masked_fill(~kept, float("-inf"))
    top = torch.where(some, t.amax(1, keepdim=True), torch.zeros_like(t[:, :1]))
    e = (t - top).exp()
    mass = torch.where(some, e.sum(1, keepdim=True), torch.ones_like(top))
    p = e / mass
    logp = torch.where(p > 0, t - top - mass.log(), torch.zeros_like(t))
    x = z / c["temperature"]
    m = x.amax(1, keepdim=True)
    q = (x - m).exp()
    total = q.sum(1, keepdim=True)
    logq = x.gather(1, idx.clamp(min=0)) - m - total.log()
    kd = c["kd"] * c["temperature"]
    loss = kd * c["temperature"] * (p * (logp - torch.where(kept, logq, torch.zeros_like(logq)))).sum(1)
    dz = None
    if c["train"]:
        dz = q.mul_(kd / total) * some
        dz.scatter_add_(1, idx.clamp(min=0), -kd * p)
    if c["ce"] > 0:
        r = torch.arange(c["rows"], device=z.device)
        has = (r % c["seq"] != c["seq"] - 1)[:, None]
        target = st["tokens"][1:].long()[:, None]
        m = z.amax(1, keepdim=True)
        q = (z - m).exp()
        total = q.sum(1, keepdim=True)
        loss = loss + (c["ce"] * (m + total.log() - z.gather(1, target)) * has).squeeze(1)
        if c["train"]:
            dz += q.mul_(c["ce"] / total * has)
            dz.scatter_add_(1, target, -c["ce"] * has.float())
    return {"loss": loss, "dz": dz.bfloat16()} if c["train"] else {"loss": loss}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own_attention(st):
    from micro_pipeline_re_gb300 import binding as b
    c, lib = st["case"], b.lib()
    n, s, h, kv = c["nseq"], c["seq"], c["heads"], c["kv_heads"]
    buf = st.get("buf")
    if buf is None:  # the program's own buffers
        buf = st["buf"] = {"o": torch.empty(n * s, h * HD, device="cuda", dtype=torch.bfloat16),
                           "lse": torch.empty(n * s, h, device="cuda")}
        if c["train"]:
            buf["dqkv"] = torch.empty_like(st["qkv"])
            if st["table"] is not None:
                buf["dtable"] = torch.empty_like(st["table"])
            size = lib.gpipe_op_attention_window_scratch_bytes(n, s, h, c["window"], c["sinks"], c["buckets"])
            st["scratch"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    ptr = b._ptr
    form = (n, s, h, kv, c["window"], c["sinks"], ptr(st["lens"]), ptr(st["table"]), c["buckets"], c["max_distance"],
            st["qkv"].data_ptr(), buf["o"].data_ptr())
    stream = b.current_stream()
    b._check(lib.gpipe_op_attention_window_fwd(*form, buf["lse"].data_ptr(), stream))
    if c["train"]:
        if st["table"] is not None:
            buf["dtable"].zero_()
        b._check(lib.gpipe_op_attention_window_bwd(*form, st["dout"].data_ptr(), buf["lse"].data_ptr(),
                                                   buf["dqkv"].data_ptr(), ptr(buf.get("dtable")),
                                                   st["scratch"].data_ptr(), stream))
    return buf


def _own_distill(st):
    from micro_pipeline_re_gb300 import binding as b
    c = st["case"]
    buf = st.get("buf")
    if buf is None:
        buf = st["buf"] = {"loss": torch.empty(c["rows"], device="cuda")}
        if c["train"]:
            buf["dz"] = torch.empty(c["rows"], c["vocab"], device="cuda", dtype=torch.bfloat16)
    ptr = b._ptr
    b._check(b.lib().gpipe_op_distill(1 if c["dtype"] == "bf16" else 0, c["rows"], c["vocab"], ptr(st["logits"]),
                                      c["vocab"] + c["pad"], c["topk"], ptr(st["top_idx"]), ptr(st["top_logit"]),
                                      c["temperature"], c["kd"], c["seq"], ptr(st["tokens"]), 0, c["ce"],
                                      ptr(buf["loss"]), ptr(buf.get("dz")), c["vocab"], b.current_stream()))
    return buf


def run(state):
    if state["case"]["op"] == "attention":
        return _own_attention(state) if own else _plain_attention(state)
    return _own_distill(state) if own else _plain_distill(state)


# ---------------------------------------------------------------------------
# Work, and the exact values
# ---------------------------------------------------------------------------
def _pairs(case):
    """Visible (query, key) pairs of one head over the batch."""
    total = 0
    for n in _lengths(case):
        w, s = case["window"], case["sinks"]
        near = n * (n + 1) // 2 if n <= w else w * (w + 1) // 2 + (n - w) * w
        # sinks that have left the window: query i has min(sinks, i - w + 1) of them
        m = max(0, n - w)
        total += near + (m * (m + 1) // 2 if m <= s else s * (s + 1) // 2 + (m - s) * s)
    return total


def work(case):
    if case["op"] == "attention":
        rows, h, kv = sum(_lengths(case)), case["heads"], case["kv_heads"]
        table = 4 * case["buckets"] * h
        # forward: qkv in, o and lse out; two products a pair.  Training: dout in and the gradients
        # out as well, and four more products (dP, dV, dQ, dK).
        nbytes = rows * ((h + 2 * kv) * HD * 2 + h * HD * 2 + 4 * h) + table
        flops = 2 * HD * 2 * _pairs(case) * h
        if case["train"]:
            nbytes += rows * ((h + 2 * kv) * HD * 2 + h * HD * 2) + table
            flops *= 3
        return {"bytes": nbytes, "flops": flops}
    rows, vocab = case["rows"], case["vocab"]
    nbytes = rows * vocab * (4 if case["dtype"] == "f32" else 2) + rows * (8 * case["topk"] + 4 + 4)
    softmaxes = 2 if case["ce"] > 0 else 1
    flops = rows * vocab * 4 * softmaxes  # scale, subtract the maximum, exponential, sum
    if case["train"]:
        nbytes += 2 * rows * vocab
        flops += rows * vocab * 2 * softmaxes
    return {"bytes": nbytes, "flops": flops}


def _exact_starts(buckets, max_distance):
    """Smallest distance of each bucket, in whole numbers: d >= me (max_distance / me)^(k / m) is
    d^m >= max_distance^k me^(m - k)."""
    me = buckets // 2
    m, starts = buckets - me, list(range(me))
    for k in range(m):
        want, lo, hi = max_distance ** k * me ** (m - k), me, max_distance
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if mid ** m >= want else (mid + 1, hi)
        starts.append(lo)
    return starts


def _exact_attention(case, seed):
    st = prepare(case, seed)
    n, s, h, kv = case["nseq"], case["seq"], case["heads"], case["kv_heads"]
    dev = st["qkv"].device
    zeros = dict(device=dev, dtype=torch.float64)
    qkv = st["qkv"].view(n, s, h + 2 * kv, HD)
    o, lse = torch.zeros(n, s, h, HD, **zeros), torch.full((n, s, h), float("-inf"), **zeros)
    dqkv = torch.zeros(n, s, h + 2 * kv, HD, **zeros)
    dtable = torch.zeros(max(1, case["buckets"]), h, **zeros)
    at = torch.arange(s, device=dev)
    dist = at[:, None] - at[None, :]
    hidden = (dist < 0) | ((dist >= case["window"]) & (at[None, :] >= case["sinks"]))
    if case["buckets"]:
        starts = torch.tensor(_exact_starts(case["buckets"], case["max_distance"]), device=dev)
        bucket = (torch.searchsorted(starts, at, right=True) - 1)[dist.clamp(min=0)]
    for b, length in enumerate(_lengths(case)):
        for head in range(h if length else 0):
            q = qkv[b, :length, head].double()
            k = qkv[b, :length, h + head // (h // kv)].double()
            v = qkv[b, :length, h + kv + head // (h // kv)].double()
            x = q @ k.T / 8.0
            if case["buckets"]:
                x += st["table"][:, head].double()[bucket[:length, :length]]
            x[hidden[:length, :length]] = float("-inf")
            lse[b, :length, head] = torch.logsumexp(x, 1)
            p = torch.exp(x - lse[b, :length, head, None])
            o[b, :length, head] = p @ v
            if case["train"]:
                g = st["dout"].view(n, s, h, HD)[b, :length, head].double()
                dp = g @ v.T
                ds = p * (dp - (g * o[b, :length, head]).sum(1, keepdim=True))
                dqkv[b, :length, head] += ds @ k / 8.0
                dqkv[b, :length, h + head // (h // kv)] += ds.T @ q / 8.0
                dqkv[b, :length, h + kv + head // (h // kv)] += p.T @ g
                if case["buckets"]:
                    w = torch.bincount(bucket[:length, :length].flatten(), weights=ds.flatten(),
                                       minlength=case["buckets"])
                    dtable[:, head] += w
    out = {"o": o.view(n * s, h * HD), "lse": lse.view(n * s, h)}
    if case["train"]:
        out["dqkv"] = dqkv.view(n * s, -1)
        if case["buckets"]:
            out["dtable"] = dtable
    return out


def _exact_distill(case, seed):
    st = prepare(case, seed)
    loss, dz = [], []
    temp, step = case["temperature"], max(1, (1 << 27) // case["vocab"])
    for r0 in range(0, case["rows"], step):
        z = st["logits"][r0:r0 + step, :case["vocab"]].double()
        rows = torch.arange(z.shape[0], device=z.device)
        idx = st["top_idx"][r0:r0 + step].long()
        p = torch.softmax((st["top_logit"][r0:r0 + step].double() / temp).masked_fill(idx < 0, float("-inf")), 1)
        p = torch.nan_to_num(p)  # rows without a teacher
        logq = torch.log_softmax(z / temp, 1)
        at = torch.gather(logq, 1, idx.clamp(min=0))
        one = case["kd"] * temp ** 2 * (torch.xlogy(p, p) - p * at).sum(1)
        grad = case["kd"] * temp * torch.exp(logq) * (idx >= 0).any(1, keepdim=True)
        grad.index_put_((rows[:, None].expand_as(idx), idx.clamp(min=0)), -case["kd"] * temp * p, accumulate=True)
        if case["ce"] > 0:
            logq = torch.log_softmax(z, 1)
            target = st["tokens"][r0 + 1:r0 + 1 + z.shape[0]].long()
            w = case["ce"] * ((r0 + rows) % case["seq"] != case["seq"] - 1).double()
            one -= w * logq[rows, target]
            if case["train"]:
                grad += w[:, None] * torch.exp(logq)
                grad[rows, target] -= w
        loss.append(one)
        dz.append(grad if case["train"] else None)
    return {"loss": torch.cat(loss), "dz": torch.cat(dz)} if case["train"] else {"loss": torch.cat(loss)}


def exact(case, seed):
    return (_exact_attention if case["op"] == "attention" else _exact_distill)(case, seed)
