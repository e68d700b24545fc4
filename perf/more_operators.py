"""Workloads of attention over long caches: a shared prefix, selected blocks, and eviction.

Five operators, each in a plain form (elementary torch operations in 32 bits or more) and, where ``own`` is true,
as the calls that a program makes of gqa_split_kv_gb300.binding:

  prefix   attention of a batch's new tokens, every sequence the same first prefix_len tokens and a rest of its own
  sparse   blocks of the cache selected for each new token by its scores with the blocks' mean keys, and attention
           over them
  means    the mean keys of the blocks that new tokens lie in
  weights  the attention weight that new tokens give each cached token, added to what it had
  evict    of each sequence and KV head, the tokens of the largest weights, moved together

A case is a dict of plain values; ``kind`` names its operator.
"""
import math

import numpy as np
import torch

own = False


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def listed():
    return [
        # a few chats behind one system prompt, one token each: latency
        dict(name="prefix_step", kind="prefix", batch=8, q_len=1, heads=32, kv_heads=8, dim=128, page=0, prefix=1024,
             lens="log", rest=256),
        # a full serving batch over one long document
        dict(name="prefix_batch", kind="prefix", batch=64, q_len=1, heads=64, kv_heads=8, dim=128, page=16,
             prefix=16384, lens="log", rest=2048),
        # drafted tokens of 16 sequences checked against the model, 256-wide heads
        dict(name="prefix_verify", kind="prefix", batch=16, q_len=4, heads=24, kv_heads=4, dim=256, page=32,
             prefix=8192, lens="uniform", rest=1000),
        # one long sequence, one token
        dict(name="sparse_step", kind="sparse", batch=1, q_len=1, heads=32, kv_heads=8, dim=128, page=0, block=64,
             select=32, lens="full", max_len=65536),
        # a ragged batch of long sequences
        dict(name="sparse_batch", kind="sparse", batch=16, q_len=1, heads=64, kv_heads=8, dim=128, page=32, block=64,
             select=64, lens="uniform", max_len=32768),
        # a prompt's chunk, every token its own blocks, 256-wide heads
        dict(name="sparse_chunk", kind="sparse", batch=2, q_len=250, heads=24, kv_heads=4, dim=256, page=32, block=64,
             select=16, lens="full", max_len=8192),
        # one token of each of 64 sequences
        dict(name="means_step", kind="means", batch=64, q_len=1, kv_heads=8, dim=128, page=16, block=64, lens="log",
             max_len=32768),
        # whole prompts
        dict(name="means_prompt", kind="means", batch=4, q_len=8192, kv_heads=8, dim=128, page=32, block=64,
             lens="uniform", max_len=8192),
        # a decode step of a ragged batch
        dict(name="weights_step", kind="weights", batch=16, q_len=1, heads=32, kv_heads=8, dim=128, int8=False,
             page=32, lens="uniform", max_len=8192),
        # the last 32 tokens of a long prompt look back over its int8 cache
        dict(name="weights_window", kind="weights", batch=1, q_len=32, heads=32, kv_heads=8, dim=128, int8=True,
             page=0, lens="full", max_len=32768),
        # a long prompt's cache down to a decode budget
        dict(name="evict_prompt", kind="evict", batch=1, kv_heads=8, dim=128, int8=False, page=0, keep=2048, first=4,
             recent=64, lens="full", max_len=32768),
        # a ragged int8 batch down to its budget, read back for the next chunk's prefill
        dict(name="evict_batch", kind="evict", batch=16, kv_heads=8, dim=128, int8=True, page=32, keep=1024, first=4,
             recent=128, lens="uniform", max_len=8192),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["prefix", "sparse", "means", "weights", "evict"])
    kv_heads = rng.choice([1, 2, 4, 8])
    page = rng.choice([0, 16, 32, 48, 64])
    if kind == "prefix":
        dim = rng.choice([64, 128, 128, 256])
        q_len = rng.choice([1, 1, 1, 2, 3, 5, 16])
        return dict(kind=kind, batch=_log_int(rng, 1, 48 // q_len), q_len=q_len, heads=kv_heads * rng.randint(1, 8),
                    kv_heads=kv_heads, dim=dim, page=page, prefix=_log_int(rng, 1, 12000),
                    lens=rng.choice(["full", "uniform", "log", "padded"]), rest=_log_int(rng, 16, 1500))
    if kind == "sparse":
        dim = rng.choice([64, 128, 128, 256])
        q_len = rng.choice([1, 1, 1, 2, 7, 60])
        block = rng.choice([16, 32, 64, 64, 128])
        return dict(kind=kind, batch=_log_int(rng, 1, max(1, 16 // q_len)), q_len=q_len,
                    heads=kv_heads * rng.randint(1, 8), kv_heads=kv_heads, dim=dim, page=page, block=block,
                    select=_log_int(rng, 2, 2048 // block), lens=rng.choice(["full", "uniform", "log"]),
                    max_len=_log_int(rng, 100, 20000))
    if kind == "means":
        top = _log_int(rng, 64, 8192)
        return dict(kind=kind, batch=_log_int(rng, 1, 4), q_len=_log_int(rng, 1, top), kv_heads=kv_heads,
                    dim=rng.choice([64, 128, 256 if kv_heads < 8 else 128]), page=page,
                    block=rng.choice([16, 32, 64, 128]), lens=rng.choice(["full", "uniform", "log"]), max_len=top)
    if kind == "weights":
        q_len = rng.choice([1, 1, 1, 2, 5, 16, 32])
        return dict(kind=kind, batch=_log_int(rng, 1, 16 if q_len == 1 else 2), q_len=q_len,
                    heads=kv_heads * rng.randint(1, 4 if q_len > 5 else 8), kv_heads=kv_heads,
                    dim=rng.choice([64, 128, 256 if kv_heads < 8 else 128]), int8=rng.random() < 0.5, page=page,
                    lens=rng.choice(["full", "uniform", "log"]), max_len=4 * _log_int(rng, 16, 2000))
    top = _log_int(rng, 64, 8192)
    first, recent = rng.choice([0, 1, 4]), _log_int(rng, 1, 64)
    return dict(kind=kind, batch=_log_int(rng, 1, 12), kv_heads=kv_heads, dim=rng.choice([32, 64, 128]),
                int8=rng.random() < 0.5, page=page, keep=_log_int(rng, first + recent, max(first + recent, top // 2)),
                first=first, recent=recent, lens=rng.choice(["full", "uniform", "log"]), max_len=4 * ((top + 3) // 4))


# ---------------------------------------------------------------- inputs

def _spread(case, top):
    """The batch's lengths up to top (the case's alone; prepare gives them to the sequences in an order of the
    seed's)."""
    B = case["batch"]
    if case["lens"] == "full":
        return np.full(B, top, np.int64)
    at = (np.arange(B) + 0.5) / B
    if case["lens"] in ("uniform", "padded"):
        lo = max(1, top // 32)
        return np.round(lo + (top - lo) * at).astype(np.int64)
    return np.clip(np.floor(np.exp(np.log(top) * at)), 1, top).astype(np.int64)


def _cap(case):
    """Tokens that a sequence's cache (with a shared prefix: its rest) has room for."""
    return case["rest"] if case["kind"] == "prefix" else case["max_len"]


def _lens(case):
    """Lengths; with a shared prefix those of the rests.  The new tokens are among them."""
    return np.maximum(_spread(case, _cap(case)), min(case.get("q_len", 1), _cap(case)))


def _pages(lens, page, cap, rng):
    """A shuffled pool for these lengths: page table [B, cap / page], entries past a sequence -1, and the pool's size."""
    need = -(-lens // page)
    table = np.full((len(lens), -(-cap // page)), -1, np.int32)
    order = rng.permutation(int(need.sum())).astype(np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, int(need.sum())


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=_device(), dtype=torch.float32).to(torch.bfloat16)


def _int32(a):
    return torch.from_numpy(np.asarray(a, np.int32)).to(_device())


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    dev = _device()
    s = dict(case=case)
    kind, B, H, D, page = case["kind"], case["batch"], case["kv_heads"], case["dim"], case["page"]
    lens, cap = _lens(case), _cap(case)
    rng.shuffle(lens)
    if kind == "prefix":
        return _prepare_prefix(s, lens, rng, gen)
    s["lens"] = _int32(lens)
    if page:
        table, pages = _pages(lens, page, cap, rng)
        s["table"] = _int32(table)
    rows = (pages, page) if page else (B, cap)
    for x in ("kv" if kind in ("sparse", "evict") else "k"):
        if case.get("int8"):
            s[x] = torch.randint(-127, 128, (*rows, H, D), generator=gen, device=dev, dtype=torch.int8)
            s[x + "_scale"] = torch.rand(rows[0], H, rows[1], generator=gen, device=dev) * 0.02 + 0.01
        else:
            s[x] = _normal(gen, *rows, H, D)
    if kind in ("sparse", "means"):
        s["means"] = torch.zeros(B, H, -(-cap // case["block"]), D, device=dev, dtype=torch.bfloat16)
    if kind == "sparse":
        _mean_keys(s, cap)  # the program has kept them up to date
    if kind in ("sparse", "weights"):
        s["q"] = _normal(gen, B, case["q_len"], case["heads"], D)
    if kind == "sparse":
        s["out"] = torch.empty_like(s["q"])
        s["blocks"] = torch.empty(B, case["q_len"], H, case["select"], device=dev, dtype=torch.int32)
    if kind in ("weights", "evict"):  # a few tokens hold most of the weight, many have none so far
        w = torch.rand(rows[0], H, rows[1], generator=gen, device=dev) ** 8 * 3
        s["weights"] = torch.where(w < 1e-6, torch.zeros_like(w), w)
    if kind == "weights":
        s["weights_out"] = torch.zeros_like(s["weights"])
    if kind == "evict":
        n = case["keep"]
        s["kept"] = torch.empty(B, H, n, device=dev, dtype=torch.int32)
        s["new_lens"] = torch.empty(B, device=dev, dtype=torch.int32)
        s["weights_out"] = torch.zeros(B, H, n, device=dev)
        for x in "kv":
            s[x + "_out"] = torch.zeros(B, n, H, D, device=dev, dtype=s[x].dtype)
            if case["int8"]:
                s[x + "_scale_out"] = torch.zeros(B, H, n, device=dev)
                s[x + "_back"] = torch.zeros(B, n, H, D, device=dev, dtype=torch.bfloat16)
    return s


def _prepare_prefix(s, lens, rng, gen):
    """The rests' pages come after the prefix's own; a page table's columns hold both."""
    case = s["case"]
    B, H, D, page, P, cap = (case[x] for x in ("batch", "kv_heads", "dim", "page", "prefix", "rest"))
    total = P + lens
    if case["lens"] == "padded":
        total[0] = 0  # the step has fewer sequences than its graph was captured with
    s["lens"] = _int32(total)
    if page:
        shared = P // page  # whole pages; one that the prefix only begins is each sequence's own copy
        table, pages = _pages(P + lens - shared * page, page, P - shared * page + cap, rng)
        last = _pages(np.array([P]), page, P, rng)[0][0]
        table[table >= 0] += len(last)
        s["prefix_table"] = _int32(last)
        s["table"] = _int32(np.concatenate((np.tile(last[:shared], (B, 1)), table), 1))
        for x in "kv":
            s[x] = _normal(gen, len(last) + pages, page, H, D)
    else:
        for x in "kv":
            s[x + "_prefix"] = _normal(gen, P, H, D)
            s[x] = _normal(gen, B, cap, H, D)
    s["q"] = _normal(gen, B, case["q_len"], case["heads"], D)
    s["out"] = torch.empty_like(s["q"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    from gqa_split_kv_gb300 import binding
    c = s["case"]
    kind, paged = c["kind"], c["page"] > 0
    if kind == "prefix":
        if paged:
            return binding.prefix_attn_paged(s["q"], s["k"], s["v"], s["prefix_table"], c["prefix"], s["table"],
                                             s["lens"], c["prefix"] + c["rest"], out=s["out"])
        return binding.prefix_attn_contig(s["q"], s["k_prefix"], s["v_prefix"], s["k"], s["v"], s["lens"],
                                          out=s["out"])
    if kind == "sparse":
        blocks = binding.block_select(s["q"], s["means"], s["lens"], c["block"], c["select"], first=1, recent=1,
                                      out=s["blocks"])
        if paged:
            return blocks, binding.sparse_attn_paged(s["q"], s["k"], s["v"], blocks, s["table"], s["lens"],
                                                     c["max_len"], c["block"], out=s["out"])
        return blocks, binding.sparse_attn_contig(s["q"], s["k"], s["v"], blocks, s["lens"], c["block"],
                                                  out=s["out"])
    if kind == "means":
        if paged:
            return binding.block_means_paged(s["k"], s["table"], s["lens"], c["max_len"], c["block"], c["q_len"],
                                             out=s["means"])
        return binding.block_means_contig(s["k"], s["lens"], c["block"], c["q_len"], out=s["means"])
    pages = (s["table"], s["lens"], c["max_len"]) if paged else (s["lens"],)
    if kind == "weights":
        if c["int8"]:
            call = binding.kv_weights_int8_paged if paged else binding.kv_weights_int8_contig
            return call(s["q"], s["k"], s["k_scale"], s["weights"], *pages, out=s["weights_out"])
        call = binding.kv_weights_paged if paged else binding.kv_weights_contig
        return call(s["q"], s["k"], s["weights"], *pages, out=s["weights_out"])
    to = dict(first=c["first"], recent=c["recent"], kept=s["kept"], new_lens=s["new_lens"], k_out=s["k_out"],
              v_out=s["v_out"], weights_out=s["weights_out"])
    if not c["int8"]:
        call = binding.kv_evict_paged if paged else binding.kv_evict_contig
        call(s["k"], s["v"], s["weights"], *pages, c["keep"], **to)
        return s["kept"], s["new_lens"], s["k_out"], s["v_out"], s["weights_out"]
    call = binding.kv_evict_int8_paged if paged else binding.kv_evict_int8_contig
    call(s["k"], s["v"], s["k_scale"], s["v_scale"], s["weights"], *pages, c["keep"], k_scale_out=s["k_scale_out"],
         v_scale_out=s["v_scale_out"], **to)
    back = binding.kv_read_int8_contig(s["k_out"], s["v_out"], s["k_scale_out"], s["v_scale_out"], s["new_lens"],
                                       c["keep"], k_out=s["k_back"], v_out=s["v_back"], zero_rest=True)
    return s["kept"], s["new_lens"], *back, s["weights_out"]


def _at(s, name, b, t):
    """Tokens t of sequences b (index tensors) of a cache: [..., H, D]."""
    page = s["case"]["page"]
    if not page:
        return s[name][b, t]
    return s[name][s["table"].clamp(min=0).long()[b, t // page], t % page]


def _scalars(s, name, b, t):
    """The same of one number a token and head, cache [B, H, tokens] or pool [pages, H, page]: [..., H]."""
    page = s["case"]["page"]
    if not page:
        return s[name][b, :, t]
    return s[name][s["table"].clamp(min=0).long()[b, t // page], :, t % page]


def _softmax(w, mask):
    """Over the tokens that the mask leaves; a row that it leaves nothing of is zeros."""
    w = w.masked_fill(~mask, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True).clamp(min=-1e30))
    return w / w.sum(-1, keepdim=True).clamp(min=1e-30)


def _seen(s):
    """[B, n]: how many tokens each new token sees."""
    n = s["case"]["q_len"]
    return s["lens"].long()[:, None] - n + 1 + torch.arange(n, device=s["lens"].device)


def _mean_keys(s, n):
    """Writes the means of the blocks that hold each sequence's last n tokens."""
    c = s["case"]
    block = c["block"]
    L = s["lens"].long()[:, None]
    j0 = (L - n).clamp(min=0) // block
    j = j0 + torch.arange(min(s["means"].shape[2], (n - 1) // block + 2), device=L.device)  # [B, blocks]
    j_ok = j * block < L
    t = j[..., None] * block + torch.arange(block, device=L.device)  # [B, blocks, block]
    t_ok = t < L[..., None]
    b = torch.arange(c["batch"], device=L.device)[:, None, None].expand_as(t)
    keys = _at(s, "k", b, torch.minimum(t, L[..., None] - 1)).float()
    keys = torch.where(t_ok[..., None, None], keys, torch.zeros_like(keys))
    mean = keys.sum(2) / t_ok.sum(2).clamp(min=1)[..., None, None]  # [B, blocks, H, D]
    s["means"][b[..., 0][j_ok], :, j[j_ok]] = mean.to(torch.bfloat16)[j_ok]
    return s["means"]


def _plain(s):
    c = s["case"]
    kind, H = c["kind"], c["kv_heads"]
    dev = s["lens"].device
    if kind == "means":
        return _mean_keys(s, c["q_len"])
    if kind == "prefix":
        return _plain_prefix(s)
    if kind == "sparse":
        return _plain_sparse(s)
    if kind == "weights":
        t = torch.arange(c["max_len"], device=dev)
        B, n, G = c["batch"], c["q_len"], c["heads"] // H
        L = s["lens"].long()
        tt = torch.minimum(t, (L[:, None] - 1).clamp(min=0))
        b = torch.arange(B, device=dev)[:, None].expand_as(tt)
        k = _at(s, "k", b, tt).float()  # [B, T, H, D]
        if c["int8"]:
            k = k * _scalars(s, "k_scale", b, tt)[..., None]
        q = s["q"].float().unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, H, n G, D]
        w = torch.matmul(q, k.permute(0, 2, 3, 1)) * c["dim"] ** -0.5
        mask = (t < _seen(s)[..., None])[:, None, :, None].expand(B, H, n, G, -1).flatten(2, 3)
        w = _softmax(w, mask).sum(2)  # [B, H, T]
        live = t < L[:, None]
        b, tt = b[live], tt[live]
        new = w.transpose(1, 2)[live] + _scalars(s, "weights", b, tt)
        if c["page"]:
            s["weights_out"][s["table"].long()[b, tt // c["page"]], :, tt % c["page"]] = new
        else:
            s["weights_out"][b, :, tt] = new
        return s["weights_out"]
    return _plain_evict(s)


def _plain_prefix(s):
    c = s["case"]
    B, n, H, D, P, page = c["batch"], c["q_len"], c["kv_heads"], c["dim"], c["prefix"], c["page"]
    G, dev = c["heads"] // H, s["lens"].device
    if page:
        t = torch.arange(P, device=dev)
        kp, vp = (s[x][s["prefix_table"].long()[t // page], t % page].float() for x in "kv")
        t = (P + torch.arange(c["rest"], device=dev)).expand(B, -1)
        b = torch.arange(B, device=dev)[:, None].expand_as(t)
        k, v = (_at(s, x, b, t).float() for x in "kv")
    else:
        kp, vp, k, v = (s[x].float() for x in ("k_prefix", "v_prefix", "k", "v"))
    q = s["q"].float().unflatten(2, (H, G)) * D ** -0.5  # [B, n, H, G, D]
    qh = q.permute(2, 0, 1, 3, 4).flatten(1, 3)  # [H, B n G, D]
    w0 = torch.matmul(qh, kp.permute(1, 2, 0)).unflatten(1, (B, n, G)).permute(1, 2, 0, 3, 4)  # [B, n, H, G, P]
    qb = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, H, n G, D]
    w1 = torch.matmul(qb, k.permute(0, 2, 3, 1)).unflatten(2, (n, G)).transpose(1, 2)
    w = torch.cat((w0, w1), -1)
    w = _softmax(w, (torch.arange(P + c["rest"], device=dev) < _seen(s)[..., None])[:, :, None, None])
    out = torch.matmul(w[..., :P].permute(2, 0, 1, 3, 4).flatten(1, 3), vp.transpose(0, 1))
    out = out.unflatten(1, (B, n, G)).permute(1, 2, 0, 3, 4)
    rest = torch.matmul(w[..., P:].transpose(1, 2).flatten(2, 3), v.transpose(1, 2))
    out = out + rest.unflatten(2, (n, G)).transpose(1, 2)
    return out.flatten(2, 3).to(torch.bfloat16)


def _plain_sparse(s):
    c = s["case"]
    B, n, H, block, pick = c["batch"], c["q_len"], c["kv_heads"], c["block"], c["select"]
    G, dev = c["heads"] // H, s["lens"].device
    blocks = s["means"].shape[2]
    seen = _seen(s)  # [B, n]
    q = s["q"].unflatten(2, (H, G))
    # scores next to the border of the selection need more than 32 bits
    score = torch.matmul(q.double().permute(0, 2, 1, 3, 4).flatten(2, 3), s["means"].double().transpose(2, 3))
    score = score.unflatten(2, (n, G)).amax(3).transpose(1, 2)  # [B, n, H, blocks]
    own_block = ((seen - 1) // block)[:, :, None, None]
    j = torch.arange(blocks, device=dev)
    score = torch.where((j == 0) | (j == own_block), torch.full_like(score, math.inf), score)
    score = torch.where(j <= own_block, score, torch.full_like(score, -math.inf))
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :pick]
    order = torch.where(order <= own_block, order, torch.full_like(order, blocks))
    order = torch.sort(order, -1)[0]
    if order.shape[-1] < pick:
        order = torch.nn.functional.pad(order, (0, pick - order.shape[-1]), value=blocks)
    chosen = torch.where(order < blocks, order, torch.full_like(order, -1))
    out = torch.empty(B, n, c["heads"], c["dim"], device=dev, dtype=torch.bfloat16)
    step = max(1, (1 << 27) // (H * pick * block * c["dim"]))  # new tokens at a time
    h = torch.arange(H, device=dev)[:, None]
    for b in range(B):
        for i in range(0, n, step):
            at = chosen[b, i:i + step]  # [m, H, pick]
            t = (at[..., None] * block + torch.arange(block, device=dev)).flatten(2)
            ok = (at[..., None] >= 0).expand(*at.shape, block).flatten(2) & (t < seen[b, i:i + step, None, None])
            t = t.clamp(min=0).minimum(s["lens"][b].long() - 1)
            if c["page"]:
                row, col = s["table"].long()[b, t // c["page"]], t % c["page"]
            else:
                row, col = torch.full_like(t, b), t
            k, v = (s[x][row, col, h].float() for x in "kv")  # [m, H, tokens, D]
            w = torch.matmul(q[b, i:i + step].float(), k.transpose(2, 3)) * c["dim"] ** -0.5
            w = _softmax(w, ok[:, :, None])
            out[b, i:i + step] = torch.matmul(w, v).flatten(1, 2).to(torch.bfloat16)
    return chosen.to(torch.int32), out


def _plain_evict(s):
    c = s["case"]
    B, H, keep, first, recent = c["batch"], c["kv_heads"], c["keep"], c["first"], c["recent"]
    dev = s["lens"].device
    L = s["lens"].long()[:, None]
    t = torch.arange(c["max_len"], device=dev).expand(B, -1)
    b = torch.arange(B, device=dev)[:, None]
    inside = torch.minimum(t, L - 1)
    w = _scalars(s, "weights", b.expand_as(t), inside).transpose(1, 2)  # [B, H, T]
    forced = ((t < first) | (t >= L - recent))[:, None]
    rank = torch.where(forced, torch.full_like(w, math.inf), w)
    rank = torch.where((t < L)[:, None], rank, torch.full_like(w, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :keep]
    order = torch.where(order < L[..., None], order, torch.full_like(order, c["max_len"]))
    order = torch.sort(order, -1)[0]
    if order.shape[-1] < keep:
        order = torch.nn.functional.pad(order, (0, keep - order.shape[-1]), value=c["max_len"])
    ok = order < c["max_len"]
    src = torch.where(ok, order, torch.zeros_like(order))  # [B, H, keep]
    h = torch.arange(H, device=dev)[:, None]
    bb = b[..., None].expand_as(src)
    if c["page"]:
        row, col = s["table"].clamp(min=0).long()[bb, src // c["page"]], src % c["page"]
    else:
        row, col = bb, src
    got = []
    for x in "kv":
        y = s[x][row, col, h].float()
        if c["int8"]:
            y = y * s[x + "_scale"][row, h, col][..., None]
        got.append(torch.where(ok[..., None], y, torch.zeros_like(y)).transpose(1, 2).to(torch.bfloat16))
    moved = s["weights"][row, h, col]
    moved = torch.where(ok, moved, torch.zeros_like(moved))
    kept = torch.where(ok, order, torch.full_like(order, -1)).to(torch.int32)
    return kept, s["lens"].clamp(max=keep), *got, moved


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind, H, page = case["kind"], case["kv_heads"], case["page"]
    lens = s["lens"].tolist()
    dev = s["lens"].device

    def tokens(name, b, t0, t1):
        """Rows [t0, t1) of sequence b's cache, token by token of its pages."""
        if not page:
            return s[name][b, t0:t1]
        at = torch.arange(t0, t1, device=dev)
        return s[name][s["table"][b].long()[at // page], at % page]

    def numbers(name, b, t0, t1):
        """One number a token and head: [H, tokens]."""
        if not page:
            return s[name][b, :, t0:t1].double()
        at = torch.arange(t0, t1, device=dev)
        return s[name][s["table"][b].long()[at // page], :, at % page].double().T

    def values(name, b, t0, t1):
        y = tokens(name, b, t0, t1).double()
        return y * numbers(name + "_scale", b, t0, t1).T[..., None] if case.get("int8") else y

    if kind == "means":
        means = s["means"].double()
        for b, L in enumerate(lens):
            for j in range(max(L - case["q_len"], 0) // case["block"], -(-L // case["block"])):
                t0 = j * case["block"]
                means[b, :, j] = values("k", b, t0, min(L, t0 + case["block"])).mean(0)
        return means
    if kind == "evict":
        return _exact_evict(s, lens, values, numbers)
    n = case["q_len"]
    G = case["heads"] // H
    scale = case["dim"] ** -0.5
    if kind == "weights":
        out = s["weights_out"].double()
        for b, L in enumerate(lens):
            k, new = values("k", b, 0, L), numbers("weights", b, 0, L)
            for i in range(n):
                m = L - n + 1 + i
                if m > 0:
                    z = torch.einsum("hgd,thd->hgt", s["q"][b, i].double().unflatten(0, (H, G)), k[:m]) * scale
                    new[:, :m] += _weights(z).sum(1)
            if page:
                at = torch.arange(L, device=dev)
                out[s["table"][b].long()[at // page], :, at % page] = new.T
            else:
                out[b, :, :L] = new
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    if kind == "prefix":
        P = case["prefix"]
        if page:
            at = torch.arange(P, device=dev)
            shared = [s[x][s["prefix_table"].long()[at // page], at % page] for x in "kv"]
        else:
            shared = [s["k_prefix"], s["v_prefix"]]
        for b, L in enumerate(lens):
            if L <= 0:
                continue
            own_rows = [tokens(x, b, P, L) if page else s[x][b, :max(L - P, 0)] for x in "kv"]
            k, v = (torch.cat(x).double() for x in zip(shared, own_rows))
            for i in range(n):
                m = L - n + 1 + i
                if m > 0:
                    z = torch.einsum("hgd,thd->hgt", s["q"][b, i].double().unflatten(0, (H, G)), k[:m]) * scale
                    out[b, i] = torch.einsum("hgt,thd->hgd", _weights(z), v[:m]).flatten(0, 1)
        return out
    block, pick = case["block"], case["select"]
    chosen = np.full(s["blocks"].shape, -1, np.int32)
    for b, L in enumerate(lens):
        k, v, means = values("k", b, 0, L), values("v", b, 0, L), s["means"][b].double()
        for i in range(n):
            last = L - n + i
            if last < 0:
                continue
            score = torch.einsum("hgd,hjd->hgj", s["q"][b, i].double().unflatten(0, (H, G)),
                                 means[:, :last // block + 1]).amax(1).cpu().numpy()
            for h in range(H):
                must = sorted({0, last // block})[:pick]
                rest = [j for j in np.argsort(-score[h], kind="stable").tolist() if j not in must]
                mine = sorted(must + rest[:pick - len(must)])
                chosen[b, i, h, :len(mine)] = mine
                t = torch.cat([torch.arange(j * block, min((j + 1) * block, last + 1)) for j in mine]).to(dev)
                z = s["q"][b, i, h * G:(h + 1) * G].double() @ k[t, h].T * scale
                out[b, i, h * G:(h + 1) * G] = _weights(z) @ v[t, h]
    return torch.from_numpy(chosen).to(dev), out


def _exact_evict(s, lens, values, numbers):
    c = s["case"]
    keep, dev = c["keep"], s["lens"].device
    kept = np.full(s["kept"].shape, -1, np.int32)
    k, v = (torch.zeros(s[x + "_out"].shape, dtype=torch.float64, device=dev) for x in "kv")
    moved = torch.zeros(s["weights_out"].shape, dtype=torch.float64, device=dev)
    for b, L in enumerate(lens):
        kb, vb, wb = values("k", b, 0, L), values("v", b, 0, L), numbers("weights", b, 0, L)
        host = wb.cpu().numpy()
        for h in range(c["kv_heads"]):
            if L <= keep:
                mine = np.arange(L)
            else:
                lo, hi = c["first"], L - c["recent"]
                best = np.argsort(-host[h, lo:hi], kind="stable")[:keep - c["first"] - c["recent"]] + lo
                mine = np.sort(np.concatenate((np.arange(lo), best, np.arange(hi, L))))
            kept[b, h, :len(mine)] = mine
            at = torch.from_numpy(mine).to(dev)
            k[b, :len(mine), h], v[b, :len(mine), h], moved[b, h, :len(mine)] = kb[at, h], vb[at, h], wb[h, at]
    new_lens = torch.tensor([min(L, keep) for L in lens], dtype=torch.int32, device=dev)
    return torch.from_numpy(kept).to(dev), new_lens, k, v, moved


def _weights(z):
    """Softmax weights of the scores z."""
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


# ---------------------------------------------------------------- what one pass cannot do without

def work(case):
    kind, H, D = case["kind"], case["kv_heads"], case["dim"]
    lens = _lens(case)
    B, n = case["batch"], case.get("q_len", 1)
    if kind == "means":
        touched = np.minimum(lens, n + (lens - n) % case["block"]) if n < lens.max() else lens
        count = -(-touched // case["block"])
        return dict(bytes=2 * H * D * int(touched.sum() + count.sum()), flops=H * D * int(touched.sum()))
    if kind == "evict":
        row = (D + 4) if case["int8"] else 2 * D
        cells = H * int(np.minimum(lens, case["keep"]).sum())
        back = 2 * cells * (row + 2 * D) if case["int8"] else 0  # read once more, bf16 out
        return dict(bytes=H * int(lens.sum()) * 4 + cells * (2 * 2 * row + 4 + 4) + back, flops=H * int(lens.sum()))
    Hq = case["heads"]
    io = 2 * 2 * B * n * Hq * D
    if kind == "weights":
        row = (D + 4) if case["int8"] else 2 * D
        seen = sum(int(np.maximum(lens - n + 1 + i, 0).sum()) for i in range(n))
        return dict(bytes=H * int(lens.sum()) * (row + 8) + io // 2, flops=2 * Hq * seen * D)
    if kind == "prefix":
        if case["lens"] == "padded":  # one of them is empty
            lens = np.sort(lens)[1:] if B > 1 else lens[:0]
        P = case["prefix"]
        seen = sum(int((P + lens - n + 1 + i).sum()) for i in range(n))
        return dict(bytes=2 * 2 * H * D * (P + int(lens.sum())) + io, flops=4 * Hq * D * seen)
    block, pick = case["block"], case["select"]
    last = np.maximum(lens[:, None] - n + np.arange(n), 0)  # [B, n]
    visible = last // block + 1
    read = np.where(visible <= pick, last + 1, (pick - 1) * block + last % block + 1)
    keys = np.minimum(lens, read.sum(1))  # of all its new tokens together, a sequence's tokens at most
    return dict(bytes=2 * 2 * H * D * int(keys.sum()) + 2 * H * D * int(visible.max(1).sum()) + io
                + 4 * B * n * H * pick,
                flops=4 * Hq * D * int(read.sum()) + 2 * Hq * D * int(visible.sum()))
