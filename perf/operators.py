"""Workloads of the cache-side operators and of latent attention.

Five operators, each in a plain form (elementary torch operations in 32 bits or more) and, where ``own`` is true,
as the calls that a program makes of gqa_split_kv_gb300.binding:

  rope    rotary positions of a batch of tokens' heads, or the gradient through them
  write   new tokens' keys (rotated) and values into a cache, then those tokens read back
  read    a cache's tokens as contiguous bf16 keys and values
  latent  attention of a few new tokens over a cache of one shared latent vector a token (absorbed form)
  expand  causal prefill over keys and values expanded from the latent vectors (expanded form)

A case is a dict of plain values; ``kind`` names its operator.
"""
import math

import numpy as np
import torch

own = False

PE = 64  # rotated elements that every head of latent attention shares


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def listed():
    return [
        # a decode step of 64 sequences: the step's 64 query heads
        dict(name="rope_step", kind="rope", tokens=64, heads=64, dim=128, rot=128, offset=0, interleaved=False,
             backward=False, dtype="bf16", scaling="none", max_pos=32768),
        # a 4096-token prompt's queries far into a context that was lengthened by parts
        dict(name="rope_prompt", kind="rope", tokens=4096, heads=32, dim=128, rot=128, offset=0, interleaved=True,
             backward=False, dtype="bf16", scaling="by_parts", max_pos=1 << 20),
        # the gradient of a training step through a quarter of 256-wide heads, in fp32
        dict(name="rope_grad_part", kind="rope", tokens=8192, heads=24, dim=256, rot=64, offset=0, interleaved=False,
             backward=True, dtype="f32", scaling="none", max_pos=8192),
        # one token of each of 64 sequences into an int8 page pool
        dict(name="write_step_int8", kind="write", batch=64, q_len=1, kv_heads=8, dim=128, rot=128, interleaved=False,
             int8=True, page=16, lens="log", max_len=32768),
        # a prefill chunk of 4 sequences into an int8 page pool
        dict(name="write_chunk_int8", kind="write", batch=4, q_len=1024, kv_heads=8, dim=128, rot=128,
             interleaved=False, int8=True, page=32, lens="full", max_len=8192),
        # a ragged int8 batch back to bf16, for the next chunk's prefill
        dict(name="read_batch_int8", kind="read", batch=16, kv_heads=8, dim=128, int8=True, page=32, lens="uniform",
             max_len=8192),
        # one contiguous int8 sequence with 256-wide heads
        dict(name="read_one_int8", kind="read", batch=1, kv_heads=4, dim=256, int8=True, page=0, lens="full",
             max_len=4096),
        # one sequence, few heads (one share of a model cut over several cards): latency
        dict(name="latent_step", kind="latent", batch=1, q_len=1, heads=16, latent=512, page=0, lens="full",
             max_len=4096),
        # all 128 heads over a ragged paged batch: as many operations a byte as the card has
        dict(name="latent_batch", kind="latent", batch=16, q_len=1, heads=128, latent=512, page=32, lens="uniform",
             max_len=8192),
        # the mixed serving batch: lengths from 1 to 32768
        dict(name="latent_mixed", kind="latent", batch=64, q_len=1, heads=64, latent=512, page=16, lens="log",
             max_len=32768),
        # a whole 4096-token prompt
        dict(name="expand_prompt", kind="expand", batch=1, q_len=4096, heads=32, dim=128, lens="full", max_len=4096),
        # a ragged chunk after cached prefixes
        dict(name="expand_chunk", kind="expand", batch=4, q_len=500, heads=16, dim=128, lens="uniform", max_len=3000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["rope", "write", "read", "latent", "expand"])
    if kind == "rope":
        dim = rng.choice([32, 64, 128, 192, 256])
        rot = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= dim])
        tokens = _log_int(rng, 1, 8192)
        return dict(kind=kind, tokens=tokens, heads=_log_int(rng, 1, 48), dim=dim, rot=rot,
                    offset=rng.choice([0, dim - rot]), interleaved=rng.random() < 0.5, backward=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "f16", "f32"]) if tokens * dim < 2**20 else "bf16",
                    scaling=rng.choice(["none", "linear", "base", "by_parts"]), max_pos=_log_int(rng, 64, 1 << 20))
    if kind == "write":
        dim = rng.choice([32, 64, 128, 256])
        page = rng.choice([0, 16, 32, 48, 64])
        q_len = _log_int(rng, 1, 1024)
        top = 4 * _log_int(rng, 256, 2048)
        batch = _log_int(rng, 1, max(1, min(64, 4096 // q_len, 65536 // top)))
        return dict(kind=kind, batch=batch, q_len=q_len, kv_heads=rng.choice([1, 2, 4, 8]), dim=dim,
                    rot=rng.choice([0, dim // 2, dim]), interleaved=rng.random() < 0.5, int8=rng.random() < 0.7,
                    page=page, lens=rng.choice(["full", "uniform", "log"]), max_len=top)
    if kind == "read":
        page = rng.choice([0, 16, 32, 48, 64])
        return dict(kind=kind, batch=_log_int(rng, 1, 16), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([32, 64, 128]), int8=page == 0 or rng.random() < 0.7, page=page,
                    lens=rng.choice(["full", "uniform", "log"]), max_len=4 * _log_int(rng, 16, 2048))
    if kind == "latent":
        q_len = rng.choice([1, 1, 1, 2, 3, 7])
        return dict(kind=kind, batch=_log_int(rng, 1, 24), q_len=q_len, heads=_log_int(rng, 1, 128 // q_len),
                    latent=rng.choice([128, 256, 512, 512]), page=rng.choice([0, 16, 32, 48, 64]),
                    lens=rng.choice(["full", "uniform", "log"]), max_len=_log_int(rng, 17, 6000))
    return dict(kind=kind, batch=_log_int(rng, 1, 4), q_len=_log_int(rng, 1, 1000), heads=_log_int(rng, 1, 16),
                dim=rng.choice([64, 128, 128]), lens=rng.choice(["full", "uniform"]), max_len=_log_int(rng, 64, 2500))


# ---------------------------------------------------------------- inputs

def _lens(case):
    """The batch's lengths (the case's alone; prepare gives them to the sequences in an order of the seed's)."""
    B, top = case["batch"], case["max_len"]
    if case["lens"] == "full":
        return np.full(B, top, np.int64)
    at = (np.arange(B) + 0.5) / B
    if case["lens"] == "uniform":
        lo = max(1, top // 32)
        return np.round(lo + (top - lo) * at).astype(np.int64)
    return np.clip(np.floor(np.exp(np.log(top) * at)), 1, top).astype(np.int64)


def _inv_freq(rot, scaling):
    """Radians a position of each rotated pair, float64 (base 10000; the scaled ones stretch 4096 positions by 8)."""
    j = np.arange(rot // 2, dtype=np.float64)
    base, factor, ctx = 10000.0, 8.0, 4096
    if scaling == "base":
        base *= factor ** (rot / (rot - 2))
    w = base ** (-2.0 * j / rot)
    if scaling == "linear":
        w = w / factor
    elif scaling == "by_parts":
        turns = ctx * w / (2 * math.pi)  # over the original context: many turns stay, few are stretched
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w = w * keep + w / factor * (1.0 - keep)
    return w


def _magnitude(scaling):
    return 0.1 * math.log(8.0) + 1.0 if scaling == "by_parts" else 1.0


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


def _normal(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=_device(), dtype=torch.float32).to(dtype)


def _int8(gen, *shape):
    return torch.randint(-127, 128, shape, generator=gen, device=_device(), dtype=torch.int8)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    dev = _device()
    s = dict(case=case)
    kind = case["kind"]
    if kind == "rope":
        dt = dict(bf16=torch.bfloat16, f16=torch.float16, f32=torch.float32)[case["dtype"]]
        s["x"] = _normal(gen, case["tokens"], case["heads"], case["dim"], dtype=dt)
        s["positions"] = torch.from_numpy(rng.integers(0, case["max_pos"], case["tokens"]).astype(np.int32)).to(dev)
        s["inv_freq"] = torch.from_numpy(_inv_freq(case["rot"], case["scaling"])).to(dev)
        s["magnitude"] = _magnitude(case["scaling"])
        s["out"] = torch.empty_like(s["x"])
        return s
    lens = _lens(case)
    rng.shuffle(lens)
    B, top = case["batch"], case["max_len"]
    if kind in ("write", "latent", "expand"):
        lens = np.maximum(lens, min(case["q_len"], top))  # a chunk's tokens are among the sequence's
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(dev)
    page = case.get("page", 0)
    if page:
        table, pages = _pages(lens, page, top, rng)
        s["table"] = torch.from_numpy(table).to(dev)
    if kind in ("write", "read"):
        H, D = case["kv_heads"], case["dim"]
        rows = (pages, page) if page else (B, top)
        n = case["q_len"] if kind == "write" else int(lens.max())
        for x in "kv":
            if case["int8"]:
                s[x] = _int8(gen, *rows, H, D)
                s[x + "_scale"] = torch.rand(rows[0], H, rows[1], generator=gen, device=dev) * 0.02 + 0.01
            else:
                s[x] = _normal(gen, *rows, H, D)
            if case["int8"] or page:
                s[x + "_out"] = torch.zeros(B, n, H, D, device=dev, dtype=torch.bfloat16)
            if kind == "write":
                s[x + "_new"] = _normal(gen, B, n, H, D)
        if kind == "write":
            s["starts"] = s["lens"] - n  # the chunk's first position
            if case["rot"]:
                s["inv_freq"] = torch.from_numpy(_inv_freq(case["rot"], "none")).to(dev)
        return s
    H = case["heads"]
    if kind == "latent":
        W = case["latent"] + PE
        s["q"] = _normal(gen, B, case["q_len"], H, W)
        s["cache"] = _normal(gen, *((pages, page) if page else (B, top)), W)
        s["out"] = torch.empty(B, case["q_len"], H, case["latent"], device=dev, dtype=torch.bfloat16)
        return s
    D = case["dim"]
    s["q"] = _normal(gen, B, case["q_len"], H, D + PE)
    kv = _normal(gen, B, top, H, 2 * D)  # one product expands a token's keys and values side by side
    s["k"], s["v"] = kv[..., :D], kv[..., D:]
    s["k_rope"] = _normal(gen, B, top, PE)
    s["out"] = torch.empty(B, case["q_len"], H, D, device=dev, dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    from gqa_split_kv_gb300 import binding
    c = s["case"]
    kind = c["kind"]
    if kind == "rope":
        return binding.rope_apply(s["x"], s["positions"], s["inv_freq"], offset=c["offset"],
                                  interleaved=c["interleaved"], magnitude=s["magnitude"], backward=c["backward"],
                                  out=s["out"])
    if kind == "write":
        rope = dict(inv_freq=s["inv_freq"], interleaved=c["interleaved"]) if c["rot"] else {}
        if c["int8"] and c["page"]:
            binding.kv_write_int8_paged(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scale"], s["v_scale"],
                                        s["table"], s["lens"], c["max_len"], **rope)
            return binding.kv_read_int8_paged(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                                              c["max_len"], c["q_len"], starts=s["starts"], k_out=s["k_out"],
                                              v_out=s["v_out"])
        if c["int8"]:
            binding.kv_write_int8_contig(s["k_new"], s["v_new"], s["k"], s["v"], s["k_scale"], s["v_scale"],
                                         s["lens"], **rope)
            return binding.kv_read_int8_contig(s["k"], s["v"], s["k_scale"], s["v_scale"], s["lens"], c["q_len"],
                                               starts=s["starts"], k_out=s["k_out"], v_out=s["v_out"])
        if c["page"]:
            binding.kv_write_paged(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lens"], c["max_len"],
                                   **rope)
            return binding.kv_read_paged(s["k"], s["v"], s["table"], s["lens"], c["max_len"], c["q_len"],
                                         starts=s["starts"], k_out=s["k_out"], v_out=s["v_out"])
        binding.kv_write_contig(s["k_new"], s["v_new"], s["k"], s["v"], s["lens"], **rope)
        return s["k"], s["v"]
    if kind == "read":  # the whole output, whatever an earlier pass left in it
        n = s["k_out"].shape[1]
        kw = dict(k_out=s["k_out"], v_out=s["v_out"], zero_rest=True)
        if c["int8"] and c["page"]:
            return binding.kv_read_int8_paged(s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                                              c["max_len"], n, **kw)
        if c["int8"]:
            return binding.kv_read_int8_contig(s["k"], s["v"], s["k_scale"], s["v_scale"], s["lens"], n, **kw)
        return binding.kv_read_paged(s["k"], s["v"], s["table"], s["lens"], c["max_len"], n, **kw)
    if kind == "latent":
        if c["page"]:
            return binding.latent_attn_paged(s["q"], s["cache"], s["table"], s["lens"], c["max_len"],
                                             scale=_scale(c), out=s["out"])
        return binding.latent_attn_contig(s["q"], s["cache"], s["lens"], scale=_scale(c), out=s["out"])
    return binding.latent_prefill_contig(s["q"], s["k"], s["k_rope"], s["v"], s["lens"], scale=_scale(c),
                                         out=s["out"])


def _scale(case):
    """One over the root of a head's width before it was absorbed (128 + 64), or of the expanded head's."""
    return (case.get("dim", 128) + PE) ** -0.5


def _rotate(x, positions, inv_freq, offset, interleaved, magnitude, sign):
    """x [..., H, D] in 32 bits, positions [...]: the rotated heads. Angles in 64 bits."""
    rot = 2 * inv_freq.numel()
    angle = positions.double()[..., None] * inv_freq
    cos = (torch.cos(angle) * magnitude).float()[..., None, :]
    sin = (torch.sin(angle) * (magnitude * sign)).float()[..., None, :]
    part = x[..., offset:offset + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rot // 2], part[..., rot // 2:])
    y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1 if interleaved else -2).flatten(-2)
    return torch.cat((x[..., :offset], y, x[..., offset + rot:]), -1)


def _rows(s, name, page):
    """A cache as [B, tokens, ...]: itself, or its pages in the table's order (entries of no page read page 0)."""
    return s[name][s["table"].clamp(min=0).long()].flatten(1, 2) if page else s[name]


def _softmax(w, mask):
    """Over the tokens that the mask leaves; a row that it leaves nothing of is zeros."""
    w = w.masked_fill_(~mask, -math.inf)
    w = torch.exp_(w.sub_(w.amax(-1, keepdim=True).clamp(min=-1e30)))
    return w.div_(w.sum(-1, keepdim=True).clamp(min=1e-30))


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "rope":
        y = _rotate(s["x"].float(), s["positions"], s["inv_freq"], c["offset"], c["interleaved"], s["magnitude"],
                    -1.0 if c["backward"] else 1.0)
        return y.to(s["x"].dtype)
    page = c.get("page", 0)
    if kind == "write":
        n = c["q_len"]
        at = s["starts"].long()[:, None] + torch.arange(n, device=s["lens"].device)  # [B, n]: the chunk's positions
        b = torch.arange(c["batch"], device=at.device)[:, None].expand_as(at)
        row, col = (s["table"].long()[b, at // page], at % page) if page else (b, at)
        for x in "kv":
            new = s[x + "_new"].float()
            if x == "k" and c["rot"]:
                new = _rotate(new, at, s["inv_freq"], 0, c["interleaved"], 1.0, 1.0)
            if c["int8"]:
                top = new.abs().amax(-1)
                scale = torch.where(top > 0, top / 127.0, torch.ones_like(top))
                s[x][row, col] = torch.round(new / scale[..., None]).clamp(-127, 127).to(torch.int8)
                s[x + "_scale"][row, :, col] = scale
            else:
                s[x][row, col] = new.to(torch.bfloat16)
        if c["int8"]:
            return tuple((s[x][row, col].float() * s[x + "_scale"][row, :, col][..., None]).to(torch.bfloat16)
                         for x in "kv")
        return tuple(s[x][row, col] if page else s[x] for x in "kv")
    if kind == "read":
        n = s["k_out"].shape[1]
        live = (torch.arange(n, device=s["lens"].device) < s["lens"][:, None])[..., None, None]
        got = []
        for x in "kv":
            y = _rows(s, x, page)[:, :n].float()
            if c["int8"]:
                sc = s[x + "_scale"]
                sc = sc[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2) if page else sc
                y = y * sc[..., :n].transpose(1, 2)[..., None]
            got.append(torch.where(live, y, torch.zeros_like(y)).to(torch.bfloat16))
        return tuple(got)
    H, n = c["heads"], c["q_len"]
    t = torch.arange(c["max_len"], device=s["lens"].device)
    seen = s["lens"].long()[:, None] - n + 1 + torch.arange(n, device=t.device)  # [B, n]: the tokens each query sees
    mask = t < seen[..., None]  # [B, n, tokens]
    if kind == "latent":
        rows = _rows(s, "cache", page)[:, :c["max_len"]].float()
        w = torch.matmul(s["q"].float().flatten(1, 2), rows.transpose(1, 2)) * _scale(c)  # [B, n H, tokens]
        w = _softmax(w.unflatten(1, (n, H)), mask[:, :, None]).flatten(1, 2)
        return torch.matmul(w, rows[..., :c["latent"]]).unflatten(1, (n, H)).to(torch.bfloat16)
    D = c["dim"]
    q = s["q"].float().transpose(1, 2)  # [B, H, n, D + PE]
    w = torch.matmul(q[..., :D], s["k"].float().permute(0, 2, 3, 1))
    w = w + torch.matmul(q[..., D:], s["k_rope"].float().transpose(1, 2)[:, None])
    w = _softmax(w * _scale(c), mask[:, None])
    return torch.matmul(w, s["v"].float().transpose(1, 2)).transpose(1, 2).to(torch.bfloat16)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "rope":
        return _exact_rotation(s["x"].double(), s["positions"], s["inv_freq"], case["offset"], case["interleaved"],
                               s["magnitude"], case["backward"])
    lens = s["lens"].tolist()

    def tokens(name, b, t0, t1):
        """Rows [t0, t1) of sequence b's cache, token by token of its pages."""
        if not case.get("page"):
            return s[name][b, t0:t1]
        at = torch.arange(t0, t1, device=s["lens"].device)
        return s[name][s["table"][b].long()[at // case["page"]], at % case["page"]]

    def values(name, b, t0, t1):
        y = tokens(name, b, t0, t1).double()
        if not case["int8"]:
            return y
        sc = s[name + "_scale"]
        if not case["page"]:
            return y * sc[b, :, t0:t1].double().T[..., None]
        at = torch.arange(t0, t1, device=sc.device)
        return y * sc[s["table"][b].long()[at // case["page"]], :, at % case["page"]].double()[..., None]

    if kind == "read":
        out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device=s["lens"].device) for _ in "kv"]
        for b, L in enumerate(lens):
            for o, name in zip(out, "kv"):
                o[b, :L] = values(name, b, 0, L)
        return tuple(out)
    if kind == "write":
        n, got = case["q_len"], []
        for name in "kv":
            x = s[name + "_new"].double()
            if name == "k" and case["rot"]:
                at = s["lens"].long()[:, None] - n + torch.arange(n, device=x.device)
                x = _exact_rotation(x, at, s["inv_freq"], 0, case["interleaved"], 1.0, False)
            if case["int8"]:
                step = x.abs().amax(-1, keepdim=True) / 127
                step = torch.where(step > 0, step, torch.ones_like(step))
                x = torch.round(x / step) * step
            if not case["int8"] and not case["page"]:  # the whole cache comes back
                whole = s[name].double()
                for b, L in enumerate(lens):
                    whole[b, L - n:L] = x[b]
                x = whole
            got.append(x)
        return tuple(got)
    n, H = case["q_len"], case["heads"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["lens"].device)
    for b, L in enumerate(lens):
        q = s["q"][b].double()
        last = L - n + torch.arange(n, device=q.device)  # the last token that each query sees
        hide = torch.arange(L, device=q.device)[None] > last[:, None]
        if kind == "latent":
            c = tokens("cache", b, 0, L).double()
            z = torch.einsum("ihw,tw->iht", q, c) * _scale(case)
            out[b] = torch.einsum("iht,tr->ihr", _weights(z, hide[:, None]), c[:, :case["latent"]])
        else:
            D = case["dim"]
            for h in range(H):
                key = torch.cat((s["k"][b, :L, h], s["k_rope"][b, :L]), -1).double()
                z = q[:, h] @ key.T * _scale(case)
                out[b, :, h] = _weights(z, hide) @ s["v"][b, :L, h].double()
    return out


def _weights(z, hide):
    """Softmax weights of the scores z, none where hide; zeros in a row with nothing else."""
    none = hide.all(-1, keepdim=True)
    z = torch.where(hide & ~none, torch.full_like(z, -math.inf), z)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    return torch.where(none, torch.zeros_like(e), e / e.sum(-1, keepdim=True))


def _exact_rotation(x, positions, inv_freq, offset, interleaved, magnitude, backward):
    """Each pair as a complex number times magnitude exp(i p w), or its conjugate."""
    rot = 2 * inv_freq.numel()
    j = torch.arange(rot // 2, device=x.device)
    a, b = (offset + 2 * j, offset + 2 * j + 1) if interleaved else (offset + j, offset + rot // 2 + j)
    turn = torch.polar(torch.full_like(inv_freq, magnitude).expand(*positions.shape, -1),
                       positions.double()[..., None] * inv_freq)
    turn = (turn.conj() if backward else turn)[..., None, :]
    z = torch.complex(x[..., a], x[..., b]) * turn
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


# ---------------------------------------------------------------- what one pass cannot do without

def work(case):
    kind = case["kind"]
    if kind == "rope":
        n = case["tokens"] * case["heads"]
        size = 4 if case["dtype"] == "f32" else 2
        return dict(bytes=2 * n * case["dim"] * size + 4 * case["tokens"], flops=3 * n * case["rot"])
    lens = _lens(case)
    if kind == "write":  # bf16 in, the cache's type out; the chunk once more in, bf16 out
        n = 2 * case["batch"] * case["q_len"] * case["kv_heads"]
        cell = (case["dim"] + 4) if case["int8"] else 2 * case["dim"]
        back = case["int8"] or case["page"] > 0
        return dict(bytes=n * (2 * case["dim"] + cell + (cell + 2 * case["dim"] if back else 0)),
                    flops=n * case["dim"] * (5 if case["int8"] else 2))
    if kind == "read":
        n = 2 * int(lens.sum()) * case["kv_heads"]
        cell = (case["dim"] + 4) if case["int8"] else 2 * case["dim"]
        return dict(bytes=n * (cell + 2 * case["dim"]), flops=n * case["dim"])
    n, H, B = case["q_len"], case["heads"], case["batch"]
    lens = np.maximum(lens, min(n, case["max_len"]))
    seen = sum(int(np.maximum(lens - n + 1 + i, 0).sum()) for i in range(n))  # (query, visible token) pairs
    if kind == "latent":
        R = case["latent"]
        return dict(bytes=2 * (int(lens.sum()) * (R + PE) + B * n * H * (2 * R + PE)),
                    flops=2 * H * seen * (2 * R + PE))
    D = case["dim"]
    return dict(bytes=2 * (int(lens.sum()) * (2 * H * D + PE) + B * n * H * (2 * D + PE)),
                flops=2 * H * seen * (2 * D + PE))
