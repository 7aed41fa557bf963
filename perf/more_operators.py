"""Cases of the two ends of a language model's vocabulary, for timing and for
checking: the head's loss, which keeps no logits, and the embedding.

Head loss (op "head"), per row of hidden states h_r with target t and weight w,
over the tied matrix E [vocab, d]:
  z = h_r E^T, limited to [-clip, clip] where clip > 0, p = softmax(z),
  loss_r = w inv_count (-log p_t),
  g      = w (p - onehot(t)), 0 where the limit cut z off,
  dh_r   = inv_count g E,   dE = inv_count sum_r g_r^T h_r.
A row's target is the next token of its sequence; the last row of a sequence has
none, and rows of weight 0 count for nothing, whatever they hold.
Embedding (ops "embed_fwd", "embed_bwd"): x_r = scale E[token_r], and
dE[v] += scale sum of dx_r over the rows of token v.  A negative token is
padding: x_r = 0 and no gradient.
"""
import math

import numpy as np
import torch

own = False  # true: run() calls the library; false: plain torch


def _head(name, rows, d, vocab, seq, piece, clip, weights, grads):
    return {"name": name, "op": "head", "rows": rows, "d": d, "vocab": vocab, "seq": seq, "piece": piece, "clip": clip,
            "weights": weights, "grads": grads}


def _embed(name, backward, rows, d, vocab, dtype, tokens, padded):
    return {"name": name, "op": "embed_bwd" if backward else "embed_fwd", "rows": rows, "d": d, "vocab": vocab,
            "dtype": dtype, "tokens": tokens, "padded": padded}


def listed():
    return [
        # a handful of tokens over a toy vocabulary: launches count
        _head("head_small_train", 5, 64, 517, 5, 0, 0.0, False, "both"),
        # the log-probability of one token, as a sampler asks for it
        _head("head_score_one", 1, 1024, 32000, 512, 0, 0.0, False, "none"),
        # a micro-batch of the small language model (4 x 128 tokens)
        _head("head_lm_small_train", 512, 512, 32000, 128, 0, 0.0, False, "both"),
        # a micro-batch of the memory-scaling workload (4 x 512 tokens)
        _head("head_lm_deep_train", 2048, 1024, 32000, 512, 0, 0.0, False, "both"),
        # fine-tuning on unequal documents: prompts without weight, a padded end, clipped logits, odd sizes
        _head("head_ragged_train", 1003, 712, 50001, 59, 8192, 9.0, True, "both"),
        # evaluation of a long document over a large vocabulary
        _head("head_eval_long", 8192, 1024, 131072, 8192, 0, 0.0, False, "none"),
        # the same in training, 16384 columns of the vocabulary at a time: the most work
        _head("head_large_train", 8192, 1024, 131072, 2048, 16384, 0.0, False, "both"),
        # a short prompt's rows
        _embed("embed_small_bwd", True, 19, 64, 517, "f32", "uniform", 0.0),
        # a micro-batch of the memory-scaling workload
        _embed("embed_lm_deep_fwd", False, 2048, 1024, 32000, "f32", "uniform", 0.0),
        _embed("embed_lm_deep_bwd", True, 2048, 1024, 32000, "f32", "uniform", 0.0),
        # padded text over a large vocabulary: few tokens make up most of the rows
        _embed("embed_text_bwd", True, 16001, 1024, 131072, "bf16", "text", 0.1),
        # the whole mini-batch of the memory-scaling workload at once, as text
        _embed("embed_batch_bwd", True, 131072, 1024, 32000, "f32", "text", 0.0),
    ]


MOST = 8192 * 1024 * 131072  # rows x d x vocab of the largest head


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    vocab = _log_int(rng, 32, 131072)
    d = 8 * _log_int(rng, 8, 256)
    if rng.random() < 0.6:
        rows = _log_int(rng, 1, max(1, min(8192, MOST // (vocab * d))))
        return _head("", rows, d, vocab, _log_int(rng, 2, max(2, 2 * rows)),
                     rng.choice((0, 0, _log_int(rng, 1024, 32768))), rng.choice((0.0, 0.0, 6.0)),
                     rows >= 16 and rng.random() < 0.5, rng.choice(("both", "both", "both", "h", "none")))
    rows = _log_int(rng, 1, min(131072, 131072 * 1024 // d))
    return _embed("", rng.random() < 0.7, rows, d, vocab, rng.choice(("f32", "bf16")), rng.choice(("uniform", "text")),
                  rng.choice((0.0, 0.0, 0.3)))


# Text: the share of the k-th most frequent token goes as 1 / (k + 2.7).
def _shares(vocab):
    w = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return w / w.sum()


def _scale(case):
    return math.sqrt(case["d"])  # rows of unit variance from a table of variance 1 / d


def _inv_count(case):
    n, s = case["rows"], case["seq"]
    return 1.0 / max(1, n - n // s)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    rows, d, vocab = case["rows"], case["d"], case["vocab"]
    st = {"case": case, "emb": (randn(vocab, d) / math.sqrt(d)).bfloat16()}
    if case["op"] == "head":
        st["tokens"] = torch.randint(0, vocab, (rows + 1,), generator=g, device="cuda", dtype=torch.int32)
        # hidden states that know something of the next token, some rows more than others
        know = 4.0 + 9.0 * torch.rand(rows, 1, generator=g, device="cuda")
        st["h"] = (randn(rows, d) + know * st["emb"][st["tokens"][1:].long()].float()).bfloat16()
        st["weight"] = None
        if case["weights"]:
            u = torch.rand(rows, generator=g, device="cuda")
            st["weight"] = torch.where(u < 0.3, torch.zeros_like(u), 0.5 + u)
            st["weight"][rows - rows // 16:] = 0.0
            st["h"][rows - rows // 16:] = float("nan")  # padding: whatever was in memory
        return st
    if case["tokens"] == "uniform":
        tok = torch.randint(0, vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    else:
        cdf = torch.from_numpy(np.cumsum(_shares(vocab))).cuda()
        u = torch.rand(rows, generator=g, device="cuda", dtype=torch.float64)
        tok = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
        tok = torch.randperm(vocab, generator=g, device="cuda")[tok].to(torch.int32)
    if case["padded"] > 0.0:
        tok[rows - int(case["padded"] * rows):] = -1
    st["tokens"] = tok
    if case["op"] == "embed_bwd":
        dx = randn(rows, d)
        st["dx"] = dx if case["dtype"] == "f32" else dx.bfloat16()
        st["demb"] = randn(vocab, d) * 0.1  # what earlier micro-batches have left
        del st["emb"]
    return st


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _targets(st):
    """(targets, weights) of the rows; rows without a target have weight 0."""
    c = st["case"]
    r = torch.arange(c["rows"], device=st["h"].device)
    has = (r % c["seq"] != c["seq"] - 1).float()
    w = has if st["weight"] is None else st["weight"] * has
    return st["tokens"][1:].long(), w


def _plain_head(st):
    c = st["case"]
    target, w = _targets(st)
    h = st["h"].float().masked_fill_((w == 0)[:, None], 0.0)
    e = st["emb"].float()
    z = torch.matmul(h, e.t())
    cut = None
    if c["clip"] > 0:
        cut = z.abs() > c["clip"]
        z.clamp_(-c["clip"], c["clip"])
    m = z.amax(1, keepdim=True)
    zt = z.gather(1, target[:, None])
    z.sub_(m).exp_()
    s = z.sum(1, keepdim=True)
    a = _inv_count(c)
    loss = (w * a)[:, None] * (m - zt + s.log())
    out = {"loss": loss.squeeze(1)}
    if c["grads"] == "none":
        return out
    z *= (w * a)[:, None] / s
    z.scatter_add_(1, target[:, None], -(w * a)[:, None])
    if cut is not None:
        z.masked_fill_(cut, 0.0)
    out["dh"] = torch.matmul(z, e).bfloat16()
    if c["grads"] == "both":
        out["demb"] = torch.matmul(z.t(), h).bfloat16()
    return out


def _plain_embed_fwd(st):
    c, tok = st["case"], st["tokens"].long()
    x = st["emb"][tok.clamp(min=0)].float() * _scale(c)
    x *= (tok >= 0)[:, None]
    return {"x": x if c["dtype"] == "f32" else x.bfloat16()}


def _plain_embed_bwd(st):
    tok = st["tokens"].long()
    dx = st["dx"].float() * (_scale(st["case"]) * (tok >= 0).float())[:, None]
    st["demb"].index_add_(0, tok.clamp(min=0), dx)
    return {"demb": st["demb"]}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------
def _own_head(st):
    from micro_pipeline_re_gb300 import binding as b
    c, lib, ptr = st["case"], b.lib(), b._ptr
    rows, d, vocab = c["rows"], c["d"], c["vocab"]
    want = {"none": 0, "h": 1, "both": 3}[c["grads"]]
    buf = st.get("buf")
    if buf is None:  # the program's own buffers
        buf = st["buf"] = {"loss": torch.empty(rows, device="cuda")}
        if want & 1:
            buf["dh"] = torch.empty(rows, d, device="cuda", dtype=torch.bfloat16)
        if want & 2:
            buf["demb"] = torch.empty(vocab, d, device="cuda", dtype=torch.bfloat16)
        size = lib.gpipe_op_head_loss_scratch_bytes(rows, d, vocab, c["piece"], want)
        st["scratch"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    b._check(lib.gpipe_op_head_loss(rows, d, vocab, ptr(st["h"]), d, ptr(st["emb"]), c["seq"], ptr(st["tokens"]), 0,
                                    ptr(st["weight"]), _inv_count(c), c["clip"], c["piece"], ptr(buf["loss"]),
                                    ptr(buf.get("dh")), d, 1, ptr(buf.get("demb")), ptr(st["scratch"]),
                                    b.current_stream()))
    return buf


def _own_embed_fwd(st):
    from micro_pipeline_re_gb300 import binding as b
    c = st["case"]
    f32 = c["dtype"] == "f32"
    if "x" not in st:
        st["x"] = torch.empty(c["rows"], c["d"], device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    b._check(b.lib().gpipe_op_embedding_scaled_fwd(0 if f32 else 1, c["rows"], c["d"], c["vocab"],
                                                   b._ptr(st["tokens"]), b._ptr(st["emb"]), _scale(c), b._ptr(st["x"]),
                                                   c["d"], b.current_stream()))
    return {"x": st["x"]}


def _own_embed_bwd(st):
    from micro_pipeline_re_gb300 import binding as b
    c, lib = st["case"], b.lib()
    if "scratch" not in st:
        size = lib.gpipe_op_embedding_sorted_bwd_scratch_bytes(c["rows"], c["d"], c["vocab"])
        st["scratch"] = torch.empty(size, device="cuda", dtype=torch.uint8)
    b._check(lib.gpipe_op_embedding_sorted_bwd(0 if c["dtype"] == "f32" else 1, c["rows"], c["d"], c["vocab"],
                                               b._ptr(st["tokens"]), b._ptr(st["dx"]), c["d"], _scale(c),
                                               b._ptr(st["demb"]), b._ptr(st["scratch"]), b.current_stream()))
    return {"demb": st["demb"]}


def run(state):
    op = state["case"]["op"]
    if op == "head":
        return _own_head(state) if own else _plain_head(state)
    if op == "embed_fwd":
        return _own_embed_fwd(state) if own else _plain_embed_fwd(state)
    return _own_embed_bwd(state) if own else _plain_embed_bwd(state)


# ---------------------------------------------------------------------------
# Work, and the exact values
# ---------------------------------------------------------------------------
def work(case):
    rows, d, vocab = case["rows"], case["d"], case["vocab"]
    if case["op"] == "head":
        products = {"none": 1, "h": 2, "both": 3}[case["grads"]]
        # h, E, tokens and weights in, losses out; the gradients out as bf16
        nbytes = 2 * rows * d + 2 * vocab * d + 8 * rows + (4 * rows if case["weights"] else 0)
        nbytes += (0, 2 * rows * d, 2 * rows * d + 2 * vocab * d)[products - 1]
        return {"bytes": nbytes, "flops": products * 2 * rows * vocab * d}
    live = rows - int(case["padded"] * rows)
    es = 4 if case["dtype"] == "f32" else 2
    if case["tokens"] == "uniform":
        seen = vocab * (1.0 - (1.0 - 1.0 / vocab) ** live)
    else:
        seen = float((1.0 - (1.0 - _shares(vocab)) ** live).sum())  # expected number of different tokens
    if case["op"] == "embed_fwd":
        return {"bytes": 4 * rows + 2 * d * seen + es * d * rows, "flops": rows * d}
    return {"bytes": 4 * rows + es * d * live + 8 * d * seen, "flops": 2 * live * d}


def _exact_head(case, seed):
    st = prepare(case, seed)
    rows, d, vocab = case["rows"], case["d"], case["vocab"]
    dev = st["h"].device
    r = torch.arange(rows, device=dev)
    weight = torch.ones(rows, device=dev, dtype=torch.float64) if st["weight"] is None else st["weight"].double()
    weight = torch.where((r + 1) % case["seq"] == 0, torch.zeros_like(weight), weight) / max(1, rows - rows // case["seq"])
    e = st["emb"].double()
    loss = torch.zeros(rows, device=dev, dtype=torch.float64)
    dh = torch.zeros(rows, d, device=dev, dtype=torch.float64)
    demb = torch.zeros(vocab, d, device=dev, dtype=torch.float64)
    live = torch.nonzero(weight)[:, 0]
    step = max(1, (1 << 28) // vocab)
    for at in range(0, live.numel(), step):
        i = live[at:at + step]
        h, t, w = st["h"][i].double(), st["tokens"].long()[i + 1], weight[i]
        z = h @ e.T
        inside = None
        if case["clip"] > 0:
            inside = (z >= -case["clip"]) & (z <= case["clip"])
            z = torch.minimum(torch.maximum(z, z.new_tensor(-case["clip"])), z.new_tensor(case["clip"]))
        logp = torch.log_softmax(z, 1)
        n = torch.arange(i.numel(), device=dev)
        loss[i] = -w * logp[n, t]
        if case["grads"] == "none":
            continue
        grad = logp.exp_()
        grad[n, t] -= 1.0
        grad *= w[:, None]
        if inside is not None:
            grad *= inside
        dh[i] = grad @ e
        if case["grads"] == "both":
            demb += grad.T @ h
    out = {"loss": loss}
    if case["grads"] != "none":
        out["dh"] = dh
    if case["grads"] == "both":
        out["demb"] = demb
    return out


def _exact_embed(case, seed):
    st = prepare(case, seed)
    tok = st["tokens"].long()
    live = torch.nonzero(tok >= 0)[:, 0]
    if case["op"] == "embed_fwd":
        x = torch.zeros(case["rows"], case["d"], device=tok.device, dtype=torch.float64)
        x[live] = st["emb"].double()[tok[live]] * math.sqrt(case["d"])
        return {"x": x}
    demb = st["demb"].double()
    # rows in the order of their tokens, summed by differences of running totals at the ends of each token's rows
    order = live[torch.argsort(tok[live], stable=True)]
    if order.numel() == 0:
        return {"demb": demb}
    last = torch.nonzero(torch.diff(tok[order], append=tok.new_tensor([-2])))[:, 0]
    for c0 in range(0, case["d"], 128):
        total = torch.cumsum(st["dx"][order, c0:c0 + 128].double(), 0)[last]
        total = torch.diff(total, dim=0, prepend=torch.zeros_like(total[:1]))
        demb[tok[order[last]], c0:c0 + 128] += total * math.sqrt(case["d"])
    return {"demb": demb}


def exact(case, seed):
    return _exact_head(case, seed) if case["op"] == "head" else _exact_embed(case, seed)
