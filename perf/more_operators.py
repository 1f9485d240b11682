"""Cases and plain forms of the softmax attention that stands beside the latent-routing mixer in a hybrid stack.

Two operators that belong together, query heads in groups that share a key and value head:

* prompt: attention over whole sequences, causal or not, with its backward pass.  Per sequence, query head h and the
  key and value head g = h // (H // G):
      s_ij = scale q_i . k_j  (j <= i where it is causal),  p_ij = exp(s_ij) / sum_j exp(s_ij),  o_i = sum_j p_ij v_j,
      dv_j = sum p_ij do_i,  ds_ij = p_ij (do_i . v_j - do_i . o_i),  dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum ds_ij q_i;
* paged: a serving step.  The new tokens' keys and values go to their places in a cache of pages, and the new tokens
  attend over the cache: token i of n new ones, in a sequence of L with them, sees the first L - n + i + 1 tokens.

Forms: "prompt" (forward pass), "train" (forward and backward pass, with the rows' log-sum-exp between them) and
"paged" (one new token for every sequence up to chunks of a long prompt).  Sequences lie one behind another
("packed", rows named by offsets), in rows of a batch padded to the longest ("padded", with lengths), or are all alike ("plain").
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases

def listed():
    def seqs(name, op, B, N, H, G, d, dv, dtype, causal, layout):
        return dict(name=name, op=op, B=B, N=N, H=H, G=G, d=d, dv=dv, dtype=dtype, causal=causal, layout=layout)

    def paged(name, B, N, L, H, G, d, dv, dtype, page, layout):
        return dict(name=name, op="paged", B=B, N=N, L=L, H=H, G=G, d=d, dv=dv, dtype=dtype, page=page, layout=layout)

    return [
        # one long prompt with the long-context layer's value heads, four query heads to a key head
        seqs("prompt_long", "prompt", 1, 32768, 16, 4, 128, 128, "bf16", True, "plain"),
        # prompts of different users in one call, one behind another, from a token to some thousands
        seqs("prompt_packed", "prompt", 24, 4096, 16, 2, 64, 64, "bf16", True, "packed"),
        # an encoder over a padded classification-shaped batch, narrow keys and wider values
        seqs("prompt_both_ways", "prompt", 16, 2048, 8, 8, 32, 64, "bf16", False, "padded"),
        # a few short sequences in fp32, odd sizes: latency
        seqs("prompt_f32", "prompt", 3, 301, 6, 3, 40, 40, "f32", True, "packed"),
        # a training step at the language-model-shaped layer's batch, length and heads
        seqs("train_lm", "train", 4, 2048, 8, 8, 64, 64, "bf16", True, "plain"),
        # training on long documents, packed, wide heads in groups
        seqs("train_packed", "train", 6, 8192, 16, 4, 128, 128, "bf16", True, "packed"),
        # training in fp32 on a small padded batch
        seqs("train_f32", "train", 5, 200, 4, 2, 48, 24, "f32", False, "padded"),
        # decoding at the decode workload's batch and heads, contexts of different lengths
        paged("decode_batch", 128, 1, 8192, 16, 2, 128, 128, "bf16", 64, "plain"),
        # decoding for one user over a long context: few rows, a long axis
        paged("decode_one", 1, 1, 65536, 16, 4, 128, 128, "bf16", 16, "plain"),
        # a few users, short contexts, fp32: latency
        paged("decode_f32", 5, 1, 300, 8, 4, 64, 64, "f32", 16, "plain"),
        # some drafted tokens for each of a batch of users, checked at once, odd group
        paged("verify", 32, 6, 2048, 10, 2, 64, 64, "bf16", 32, "packed"),
        # chunks of long prompts between kept context and what comes next
        paged("chunk", 4, 1024, 16384, 16, 4, 128, 128, "bf16", 128, "packed"),
    ]


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "paged", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    G = rng.choice([1, 2, 3, 4, 8])
    H = G * rng.choice([1, 2, 3, 4, 8] if G < 8 else [1, 2, 4])
    d = rng.choice([32, 64, 64, 128, 128, 16 * rng.randint(1, 8), rng.randint(8, 128)])
    dv = d if rng.random() < 0.7 else rng.choice([16, 64, 128])
    layout = rng.choice(["plain", "packed", "packed", "padded"])
    B = _log_int(rng, 1, 32)
    if op == "paged":
        # the cost is what the new tokens' scores and the cache's bytes are
        top = (1 << 32) if dtype == "bf16" else (1 << 28)
        N = rng.choice([1, 1, _log_int(rng, 1, 16), _log_int(rng, 1, 1024)])
        L = _log_int(rng, N, max(N, min(32768, top // (B * N * H * 64), (1 << 21) // B)))
        return dict(op=op, B=B, N=N, L=L, H=H, G=G, d=d, dv=dv, dtype=dtype, page=rng.choice([16, 16, 32, 64, 128, 256, 24]),
                    layout=layout)
    pairs = ((1 << 31) if op == "prompt" else (1 << 30)) if dtype == "bf16" else (1 << 25)
    N = _log_int(rng, 1, min(8192, int(math.sqrt(pairs // (B * H)))))
    return dict(op=op, B=B, N=N, H=H, G=G, d=d, dv=dv, dtype=dtype, causal=rng.random() < 0.75, layout=layout)


def _shares(case):
    """The sequences' shares of the longest one, the same for every seed: evenly spread, shuffled by a step."""
    B = case["B"]
    if case["layout"] == "plain" and case["op"] != "paged":
        return [1.0] * B
    return [(1 + (i * 7 + 3) % B) / B if math.gcd(7, B) == 1 else (1 + (i * 11 + 3) % B) / B for i in range(B)]


def _sizes(case):
    """(new tokens, tokens in all) of every sequence."""
    share = _shares(case)
    if case["op"] != "paged":
        n = [max(1, round(case["N"] * s)) for s in share]
        return n, n
    new = [case["N"]] * case["B"] if case["layout"] == "plain" else [max(1, round(case["N"] * (0.5 + s / 2))) for s in share]
    return new, [max(a, round(case["L"] * s)) for a, s in zip(new, share)]


def work(case):
    """Inputs read once, outputs written once; the flops of the products over the scores that are not masked."""
    e = 2 if case["dtype"] == "bf16" else 4
    H, G, d, dv = case["H"], case["G"], case["d"], case["dv"]
    new, total = _sizes(case)
    rows = sum(new)
    if case["op"] == "paged":
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(new, total))
        kv = sum(total) * G * (d + dv) + sum(new) * G * (d + dv)      # the cache read, the new rows read and written there
        return {"bytes": e * (rows * H * (d + dv) + kv), "flops": 2 * pairs * H * (d + dv)}
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in new)
    one = rows * (H * (d + dv) + G * (d + dv)) * e
    if case["op"] == "prompt":
        return {"bytes": one, "flops": 2 * pairs * H * (d + dv)}
    # do in; dq, dk and dv out; the scores and four more products
    return {"bytes": one + e * rows * (H * (d + dv) + G * (d + dv)) + 4 * rows * H,
            "flops": 2 * pairs * H * (d + dv) + 2 * pairs * H * (3 * d + 2 * dv)}


# ------------------------------------------------------------------------------------ inputs

def _rows(case, new):
    """Rows of the batch's tensors: [T] packed, [B, N] otherwise."""
    return (sum(new),) if case["layout"] == "packed" else (case["B"], case["N"])


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    T = TYPES[case["dtype"]]
    B, H, G, d, dv = case["B"], case["H"], case["G"], case["d"], case["dv"]
    new, total = _sizes(case)
    lead = _rows(case, new)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(T)

    s = {"new": new, "total": total, "scale": d ** -0.5}
    # queries, keys and values are parts of one projection's rows
    width = H * d + G * (d + dv)
    x = normal(*lead, width)
    s["q"] = x[..., :H * d].unflatten(-1, (H, d))
    s["k"] = x[..., H * d:(H + G) * d].unflatten(-1, (G, d))
    s["v"] = x[..., (H + G) * d:].unflatten(-1, (G, dv))
    s["offsets"] = s["lengths"] = None
    count = torch.tensor(new, dtype=torch.int32)
    if case["layout"] == "packed":
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int32), count.cumsum(0).int()]).cuda()
    elif case["layout"] == "padded":
        s["lengths"] = count.cuda()
    if case["op"] == "train":
        s["do"] = normal(*lead, H, dv)
    if case["op"] == "paged":
        page = case["page"]
        need = [-(-t // page) for t in total]
        pages = sum(need) + 3                                       # some that are free
        s["k_pages"], s["v_pages"] = normal(pages, page, G, d), normal(pages, page, G, dv)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(max(need), device="cuda") < torch.tensor(need, device="cuda")[:, None]] = order[:sum(need)]
        s["table"] = table
        s["cached"] = torch.tensor(total, dtype=torch.int32).cuda()
    return s


def prepare(case, seed):
    return dict(_inputs(case, seed), case=dict(case))


# ------------------------------------------------------------------------------------ plain forms

MOST = 1 << 30          # scores held at once


def _span(case, i, new):
    """Where the rows of sequence i lie."""
    if case["layout"] == "packed":
        return slice(sum(new[:i]), sum(new[:i + 1]))
    return i, slice(0, new[i])


def _attend(q, k, v, scale, first, causal, do=None):
    """Attention of rows q [n, H, d], whose first is token `first`, over k and v [L, G, .]; fp32, and the gradients
    with do.  A part of the rows at a time."""
    n, H, d = q.shape
    G, L = k.shape[1], k.shape[0]
    kh, vh = k.float().permute(1, 2, 0), v.float().permute(1, 0, 2)             # [G, d, L], [G, L, dv]
    o, lse, dq = [], [], []
    dk, dv = torch.zeros_like(kh), torch.zeros_like(vh)
    step = max(1, MOST // (H * L))
    for r in range(0, n, step):
        m = min(step, n - r)
        end = min(L, first + r + m) if causal else L                            # keys behind it are seen by no row
        qh = q[r:r + m].float().permute(1, 0, 2).reshape(G, H // G * m, d)      # [G, rows, d]
        s = (torch.matmul(qh, kh[:, :, :end]) * scale).view(H, m, end)
        if causal:
            at = first + r + torch.arange(m, device=q.device)
            s.masked_fill_(torch.arange(end, device=q.device) > at[:, None], -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s.sub_(top))
        total = p.sum(-1, keepdim=True)
        p /= total
        p = p.view(G, -1, end)
        oh = torch.matmul(p, vh[:, :end])
        o.append(oh.view(H, m, -1).permute(1, 0, 2))
        lse.append((top + torch.log(total)).squeeze(-1))
        if do is not None:
            doh = do[r:r + m].float().permute(1, 0, 2).reshape(G, H // G * m, -1)
            dv[:, :end] += torch.matmul(p.transpose(1, 2), doh)
            ds = torch.matmul(doh, vh[:, :end].transpose(1, 2)).sub_((doh * oh).sum(-1, keepdim=True)).mul_(p).mul_(scale)
            dq.append(torch.matmul(ds, kh[:, :, :end].transpose(1, 2)).view(H, m, d).permute(1, 0, 2))
            dk[:, :, :end] += torch.matmul(qh.transpose(1, 2), ds)
    if do is None:
        return torch.cat(o), torch.cat(lse, 1)
    return torch.cat(o), torch.cat(lse, 1), torch.cat(dq), dk.permute(2, 0, 1), dv.permute(1, 0, 2)


def _plain_seqs(s, case):
    T, new = TYPES[case["dtype"]], s["new"]
    lead, H, G, d, dv = _rows(case, new), case["H"], case["G"], case["d"], case["dv"]
    train = case["op"] == "train"
    o = torch.zeros(*lead, H, dv, device="cuda", dtype=T)
    lse = torch.zeros((H,) + lead if len(lead) == 1 else (lead[0], H, lead[1]), device="cuda")
    grads = [torch.zeros(*lead, h, w, device="cuda", dtype=T) for h, w in ((H, d), (G, d), (G, dv))] if train else []
    for i in range(case["B"]):
        at = _span(case, i, new)
        got = _attend(s["q"][at], s["k"][at], s["v"][at], s["scale"], 0, case["causal"], s["do"][at] if train else None)
        o[at] = got[0].to(T)
        (lse[:, at] if len(lead) == 1 else lse[i, :, at[1]]).copy_(got[1])
        for g, x in zip(grads, got[2:]):
            g[at] = x.to(T)
    return [o, lse] + grads if train else o


def _plain_paged(s, case):
    """All sequences at once: rows padded to the most new tokens, keys to the longest context."""
    T, new, total = TYPES[case["dtype"]], s["new"], s["cached"].long()
    B, H, G, page = case["B"], case["H"], case["G"], case["page"]
    N, L = max(new), max(s["total"])
    if s["offsets"] is not None:
        first, n = s["offsets"][:-1].long()[:, None], s["offsets"].long().diff()[:, None]
    else:
        first = torch.arange(B, device="cuda")[:, None] * case["N"]
        n = s["lengths"].long()[:, None] if s["lengths"] is not None else torch.full((B, 1), N, device="cuda")
    i = torch.arange(N, device="cuda")
    alive = i < n                                                               # [B, N]
    row = (first + i).clamp(max=s["q"].numel() // (H * case["d"]) - 1)          # rows of the flattened tensors
    at = (total[:, None] - n + i).clamp(min=0)                                  # tokens of the sequences
    q, k, v = (s[x].flatten(0, -3) for x in "qkv")
    where = torch.gather(s["table"].long(), 1, at // page)[alive]
    s["k_pages"][where, (at % page)[alive]] = k[row[alive]]
    s["v_pages"][where, (at % page)[alive]] = v[row[alive]]
    used = s["table"].long().clamp(min=0)
    j = torch.arange(L, device="cuda")
    kh = s["k_pages"][used].flatten(1, 2)[:, :L].float().permute(0, 2, 3, 1)     # [B, G, d, L]
    vh = s["v_pages"][used].flatten(1, 2)[:, :L].float().permute(0, 2, 1, 3)     # [B, G, L, dv]
    vh = torch.where((j < total[:, None])[:, None, :, None], vh, 0.0)
    qh = q[row].float().view(B, N, G, H // G, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = (torch.matmul(qh, kh) * s["scale"]).view(B, G, N, H // G, L)
    score.masked_fill_((j > at[..., None])[:, None, :, None], -math.inf)
    p = torch.exp(score.sub_(score.amax(-1, keepdim=True)))
    p /= p.sum(-1, keepdim=True)
    out = torch.matmul(p.view(B, G, -1, L), vh).view(B, G, N, H // G, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)
    o = torch.zeros(*_rows(case, new), H, case["dv"], device="cuda", dtype=T)
    o.flatten(0, -3)[row[alive]] = out[alive].to(T)
    return o, s["k_pages"], s["v_pages"]


# ------------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return _plain_paged(s, case) if op == "paged" else _plain_seqs(s, case)
    from linear_latent_routing_gb300 import attention
    if op == "paged":
        where = dict(new_lengths=s["lengths"], offsets=s["offsets"])
        attention.append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["cached"], **where)
        o = attention.paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["cached"], scale=s["scale"], **where)
        return o, s["k_pages"], s["v_pages"]
    how = dict(causal=case["causal"], scale=s["scale"], lengths=s["lengths"], offsets=s["offsets"])
    if op == "prompt":
        return attention.prompt(s["q"], s["k"], s["v"], **how)
    # the statistics of rows that hold no token are not written
    lse = attention.prompt_lse(s["q"]) if s["lengths"] is None else attention.prompt_lse(s["q"]).zero_()
    o = attention.prompt(s["q"], s["k"], s["v"], lse=lse, **how)
    g = attention.prompt_backward(s["do"], s["q"], s["k"], s["v"], o, lse, **how)
    return [o, lse, g["q"], g["k"], g["v"]]


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """One sequence and query head after another, from the definition; gradients by reverse differentiation of it."""
    w = work(case)["flops"]
    if w > 6e12:                        # in 64 bits more than about 20 seconds
        return None
    s = _inputs(case, seed)
    new, total, H, G = s["new"], s["total"], case["H"], case["G"]
    lead, train, packed = _rows(case, new), case["op"] == "train", case["layout"] == "packed"
    f64 = dict(device="cuda", dtype=torch.float64)
    o = torch.zeros(*lead, H, case["dv"], **f64)
    lse = torch.zeros(*((H,) + lead if packed else (lead[0], H, lead[1])), **f64)
    dq, dk, dv = torch.zeros(*lead, H, case["d"], **f64), torch.zeros(*lead, G, case["d"], **f64), torch.zeros(*lead, G, case["dv"], **f64)
    start = 0
    for i, (n, L) in enumerate(zip(new, total)):
        def mine(t):
            return t[start:start + n] if packed else t[i, :n]
        q, k, v = mine(s["q"]), mine(s["k"]), mine(s["v"])
        if case["op"] == "paged":
            places = [(int(p), j) for p in s["table"][i].tolist() for j in range(case["page"])][:L]
            page, slot = (torch.tensor(x, device="cuda") for x in zip(*places))
            k, v = torch.cat([s["k_pages"][page, slot][:L - n], k]), torch.cat([s["v_pages"][page, slot][:L - n], v])
        hidden = None
        if case["op"] == "paged" or case["causal"]:
            hidden = torch.ones(n, L, device="cuda", dtype=torch.bool).triu(L - n + 1)
        for h in range(H):
            g = h // (H // G)
            leaf = [t.double().detach().requires_grad_(train) for t in (q[:, h], k[:, g], v[:, g])]
            score = leaf[0] @ leaf[1].T * s["scale"]
            if hidden is not None:
                score = score.masked_fill(hidden, -math.inf)
            out = torch.softmax(score, -1) @ leaf[2]
            mine(o)[:, h] = out.detach()
            if train:
                (lse[h, start:start + n] if packed else lse[i, h, :n]).copy_(torch.logsumexp(score, -1).detach())
                out.backward(mine(s["do"])[:, h].double())
                mine(dq)[:, h] = leaf[0].grad
                mine(dk)[:, g] += leaf[1].grad
                mine(dv)[:, g] += leaf[2].grad
        start += n
    if case["op"] == "paged":
        return o, None, None
    return [o, lse, dq, dk, dv] if train else o
