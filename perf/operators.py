"""The operators of step-by-step attention, as cases that can be timed and compared.

Four kinds of case:

* ``rope``    norms of queries and keys with the position rotation, from the
              projections' layout [B, L, H, d] to the attention's [B, H, L, d]
              (``ab_qk_norm_rope``);
* ``cache``   one step of a paged key-value cache: block tables and slot maps
              from the requests' lengths, then norm, rotation, write into the
              cache and page summaries (``ab_paged_plan``, ``ab_paged_append``);
* ``select``  the estimated share of every page in a new token's attention mass
              (``ab_paged_select``);
* ``attend``  attention of one new token per sequence over the cache: all pages,
              or the pages that ``ab_paged_topk`` keeps (``ab_attention_paged``).

``run`` computes a case in elementary torch operations, or with the library's
calls where ``own`` is true.
"""
import math

import torch

own = False

EPS = 1e-6
BF16 = torch.bfloat16


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one self-attention layer of a 480p clip (21 x 30 x 52 tokens, 40 heads): norm over the token, pairs (2i, 2i+1)
        dict(name="rope-clip480", kind="rope", B=1, H=40, L=32760, Lk=32760, d=128, norm="token", interleaved=True, pos=False),
        # a short ragged cross-attention: odd lengths, explicit positions, pairs (i, i + d/2)
        dict(name="rope-ragged", kind="rope", B=2, H=5, L=901, Lk=1333, d=64, norm="head", interleaved=False, pos=True),
        # one new token of one sequence, 40 heads: the smallest step, where latency counts
        dict(name="cache-one", kind="cache", S=1, Hq=40, Hkv=40, d=128, page=16, max_len=1500, new=1, ended=0, idle=0, norm="token",
             interleaved=True),
        # one step of 256 sequences that share the cache, some ended, some idle: the slots are padded
        dict(name="cache-step256", kind="cache", S=256, Hq=32, Hkv=8, d=128, page=16, max_len=8192, new=1, ended=9, idle=14, norm="head",
             interleaved=False),
        # prompts of very different lengths enter the cache at once
        dict(name="cache-prompts", kind="cache", S=24, Hq=32, Hkv=8, d=128, page=32, max_len=4000, new=2600, ended=3, idle=2, norm="head",
             interleaved=True),
        # few pages, one group per head: the smallest selection
        dict(name="select-small", kind="select", S=3, Hq=12, Hkv=12, d=64, page=32, max_len=1500),
        # long sequences, eight key heads with four query heads each
        dict(name="select-long", kind="select", S=48, Hq=32, Hkv=8, d=128, page=16, max_len=65536),
        # one token after 777: latency
        dict(name="attend-one", kind="attend", S=1, Hq=12, Hkv=12, d=128, page=16, max_len=777, even=True, keep=0.0, recent=0),
        # a batch of requests of very different lengths
        dict(name="attend-ragged64", kind="attend", S=64, Hq=32, Hkv=8, d=128, page=16, max_len=16384, even=False, keep=0.0, recent=0),
        # few very long sequences: work split over the length
        dict(name="attend-long", kind="attend", S=8, Hq=32, Hkv=4, d=128, page=64, max_len=131000, even=True, keep=0.0, recent=0),
        # 40 heads of their own, 11 % of the pages kept
        dict(name="attend-kept", kind="attend", S=8, Hq=40, Hkv=40, d=128, page=16, max_len=32760, even=True, keep=0.11, recent=1),
        # small heads, short sequences, lists
        dict(name="attend-kept-small", kind="attend", S=5, Hq=8, Hkv=2, d=64, page=32, max_len=2500, even=False, keep=0.2, recent=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(1, 1), (4, 4), (12, 12), (40, 40), (8, 2), (14, 2), (32, 8), (32, 4), (15, 5), (16, 1)])


def draw(rng):
    kind = rng.choice(["rope", "cache", "select", "attend", "attend"])
    d = rng.choice([64, 128])
    style = dict(norm=rng.choice(["head", "token", "none"]), interleaved=rng.random() < 0.5)
    if kind == "rope":
        L = _log(rng, 17, 32000)
        H = rng.randint(1, 40)
        return dict(kind=kind, B=1, H=H, L=L, Lk=L if rng.random() < 0.5 else _log(rng, 17, 32000), d=d, pos=rng.random() < 0.5, **style)
    Hq, Hkv = _heads(rng)
    page = rng.choice([16, 32, 64])
    S = _log(rng, 1, 200)
    if kind == "cache":
        new = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, 30000 // S))
        return dict(kind=kind, S=S, Hq=Hq, Hkv=Hkv, d=d, page=page, max_len=_log(rng, 40, 4000), new=new, ended=rng.randint(0, S // 5),
                    idle=rng.randint(0, S // 5), **style)
    if kind == "select":
        # at most the work of the longest listed selection
        top = min(65536, 48 * 65536 * 8 // (S * Hkv * (1 if page > 16 else 2)))
        return dict(kind=kind, S=S, Hq=Hq, Hkv=Hkv, d=d, page=page, max_len=_log(rng, min(100, top), max(101, top)))
    top = min(131000, 8 * 131000 * 4 // (S * Hkv))
    keep = rng.choice([0.0, 0.0, 0.05, 0.11, 0.5])
    return dict(kind=kind, S=S, Hq=Hq, Hkv=Hkv, d=d, page=page, max_len=_log(rng, min(20, top), max(21, top)), even=rng.random() < 0.3,
                keep=keep, recent=rng.randint(0, 3) if keep else 0)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _cpu_gen(seed):
    return torch.Generator().manual_seed(int(seed) * 104729 + 5)


def _requests(case):
    """(length, new tokens) of every sequence, by the case alone: lengths near max_len or spread over its logarithm, the
    longest of them max_len; -1 new tokens: the sequence has ended."""
    g = torch.Generator().manual_seed(case["S"] * 100003 + case["max_len"])
    S, top = case["S"], case["max_len"]
    u = torch.rand(S, generator=g, dtype=torch.float64)
    if case.get("even") or case["kind"] == "select":
        n = top - (u * (top // 8)).long()
    else:
        n = torch.exp(u * math.log(top)).round().long().clamp(1, top)
    n[0] = top
    new = [0] * S
    if case["kind"] == "cache":
        new = [1] * S if case["new"] == 1 else torch.randint(1, 2 * case["new"], (S,), generator=g).tolist()
        order = torch.randperm(S, generator=g).tolist()
        for s in order[:case["ended"]]:
            new[s] = -1
        for s in order[case["ended"]:case["ended"] + case["idle"]]:
            new[s] = 0
    return list(zip(n.tolist(), new))


def _tables(n_pos, d):
    """cos and sin of the rotation, fp32 of angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return a.cos().float().contiguous(), a.sin().float().contiguous()


def _weights(case, H, g):
    if case["norm"] == "none":
        return None
    shape = (case["d"],) if case["norm"] == "head" else (H, case["d"])
    return 1.0 + 0.2 * torch.randn(shape, device="cuda", generator=g)


def _cdiv(a, b):
    return -(-a // b)


def _table(lens, page, max_pages, num_pages, g):
    """Block table [S, max_pages] (0 behind a sequence's last page): distinct pages in random order, and the pages left."""
    perm = torch.randperm(num_pages, generator=g)
    table = torch.zeros(len(lens), max_pages, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        k = _cdiv(n, page)
        table[s, :k] = perm[at:at + k].to(torch.int32)
        at += k
    return table.cuda(), perm[at:].to(torch.int32)


def _randn(shape, g):
    return torch.randn(shape, device="cuda", dtype=BF16, generator=g)


def prepare(case, seed):
    g, c = _gen(seed), _cpu_gen(seed + 1)
    kind, d = case["kind"], case["d"]
    st = dict(case=case)
    if kind == "rope":
        B, H, L, Lk = case["B"], case["H"], case["L"], case["Lk"]
        if L == Lk:  # one fused projection, tokens of 3 H d values
            x = _randn((B, L, 3, H, d), g)
            st["q"], st["k"], st["v"] = x[:, :, 0], x[:, :, 1], x[:, :, 2]
        else:
            y = _randn((B, Lk, 2, H, d), g)
            st["q"], st["k"], st["v"] = _randn((B, L, H, d), g), y[:, :, 0], y[:, :, 1]
        n_pos = max(L, Lk) + 7
        st["cos"], st["sin"] = _tables(n_pos, d)
        st["wq"], st["wk"] = _weights(case, H, g), _weights(case, H, g)
        st["pos_q"] = torch.randint(0, n_pos, (B, L), device="cuda", dtype=torch.int32, generator=g) if case["pos"] else None
        st["pos_k"] = torch.randint(0, n_pos, (B, Lk), device="cuda", dtype=torch.int32, generator=g) if case["pos"] else None
        st["out"] = tuple(torch.zeros(B, H, n, d, dtype=BF16, device="cuda") for n in (L, Lk, Lk))
        return st
    S, Hq, Hkv, page = case["S"], case["Hq"], case["Hkv"], case["page"]
    requests = _requests(case)
    requests = [requests[s] for s in torch.randperm(S, generator=c).tolist()]
    lens, n_new = [n for n, _ in requests], [m for _, m in requests]
    if kind == "cache":
        tokens = sum(max(n, 0) for n in n_new)
        T = S if case["new"] == 1 else max(1, tokens)  # the slot map's length: padded in a step of single tokens
        max_pages = _cdiv(max(n + max(m, 0) for n, m in zip(lens, n_new)), page) + 1
        num_pages = sum(_cdiv(n, page) for n in lens) + _cdiv(tokens, page) + S + 5
        st["table"], left = _table(lens, page, max_pages, num_pages, c)
        free = torch.zeros(num_pages, dtype=torch.int32)
        free[:len(left)] = left
        st["free_pages"], st["free_count"] = free.cuda(), torch.tensor([len(left)], dtype=torch.int32).cuda()
        st["free_count_out"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["lens"], st["n_new"] = (torch.tensor(v, dtype=torch.int32).cuda() for v in (lens, n_new))
        st["lens_out"] = torch.zeros(S, dtype=torch.int32, device="cuda")
        st["cu_new"] = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
        st["slots"], st["positions"] = (torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
        st["T"], st["num_pages"], st["max_pages"] = T, num_pages, max_pages
        st["cos"], st["sin"] = _tables(max_pages * page, d)
        st["wq"], st["wk"] = _weights(case, Hq, g), _weights(case, Hkv, g)
        x = _randn((T, Hq + 2 * Hkv, d), g)  # the fused projection of the new tokens
        st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        st["Q"] = torch.zeros(T, Hq, d, dtype=BF16, device="cuda")
        st["K"], st["V"] = _randn((num_pages, Hkv, page, d), g), _randn((num_pages, Hkv, page, d), g)
        st["ksum"] = _randn((num_pages, Hkv, d), g)
        return st
    max_pages = _cdiv(max(lens), page)
    num_pages = sum(_cdiv(n, page) for n in lens) + 3
    st["table"], _ = _table(lens, page, max_pages, num_pages, c)
    st["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
    st["max_pages"], st["num_pages"] = max_pages, num_pages
    st["Q"] = 1.5 * torch.randn(S, Hq, d, device="cuda", generator=g)
    st["Q"] = st["Q"].to(BF16)
    if kind == "select":
        st["ksum"] = (0.8 * torch.randn(num_pages, Hkv, d, device="cuda", generator=g)).to(BF16)
        st["P"] = torch.zeros(S, Hkv, max_pages, device="cuda")
        return st
    st["K"], st["V"] = _randn((num_pages, Hkv, page, d), g), _randn((num_pages, Hkv, page, d), g)
    st["O"] = torch.zeros(S, Hq, d, dtype=BF16, device="cuda")
    if case["keep"]:
        P = torch.rand(S, Hkv, max_pages, device="cuda", generator=g) ** 6 + 1e-9
        P = P * (torch.arange(max_pages, device="cuda") < ((st["lens"] + page - 1) // page)[:, None])[:, None]
        st["P"] = (P / P.sum(-1, keepdim=True)).contiguous()
        st["idx"] = torch.zeros(S, Hkv, max_pages, dtype=torch.int32, device="cuda")
        st["count"] = torch.zeros(S, Hkv, dtype=torch.int32, device="cuda")
        st["most"] = max(min(max(int(math.floor(_keep(case) * n + 0.5)), 1), n) for n in (_cdiv(x, page) for x in lens))
    return st


def _keep(case):
    """The kept fraction as the 32-bit number that the parameters hold."""
    return torch.tensor(case["keep"], dtype=torch.float32).item()


# ------------------------------------------------------- the plain operators
def _norm_rotate(x, w, cos, sin, pos, case):
    """x [..., H, d] of tokens at positions pos [...]; fp32."""
    x = x.float()
    if case["norm"] == "head":
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    elif case["norm"] == "token":
        x = x * torch.rsqrt(x.square().mean((-2, -1), keepdim=True) + EPS) * w
    c, s = cos[pos.long()].unsqueeze(-2), sin[pos.long()].unsqueeze(-2)
    if case["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, a * s + b * c), -1)


def _run_rope(st, case):
    def side(x, w, pos, out):
        if pos is None:
            pos = torch.arange(x.shape[1], device=x.device)[None].expand(x.shape[0], -1)
        out.copy_(_norm_rotate(x, w, st["cos"], st["sin"], pos, case).transpose(1, 2))

    Q, K, V = st["out"]
    side(st["q"], st["wq"], st["pos_q"], Q)
    side(st["k"], st["wk"], st["pos_k"], K)
    V.copy_(st["v"].transpose(1, 2))
    return {"Q": Q, "K": K, "V": V}


def _run_plan(st, case):
    page, T, num_pages, max_pages = case["page"], st["T"], st["num_pages"], st["max_pages"]
    lens, n, table = st["lens"].long(), st["n_new"].long(), st["table"]
    old = (lens + page - 1) // page
    ended = n < 0
    released = torch.where(ended, old, 0)
    want = n.clamp(min=0)
    want = torch.where(lens + want > max_pages * page, 0, want)
    need = torch.where(ended, 0, (lens + want + page - 1) // page - old)
    F0 = st["free_count"].long()
    F = F0 + released.sum()
    served = (need.cumsum(0) <= F) & (want.cumsum(0) <= T)
    want, need = torch.where(served, want, 0), torch.where(served, need, 0)
    st["lens_out"].copy_(torch.where(ended, 0, lens + want))
    st["cu_new"][1:] = want.cumsum(0)
    # the list of free pages with the released ones on top
    j = torch.arange(max_pages, device=lens.device)
    back = (j < released[:, None]).flatten()
    to = torch.where(back, F0 + back.cumsum(0) - 1, num_pages)
    stack = torch.cat((st["free_pages"], st["free_pages"][:1])).scatter(0, to, table.flatten())[:num_pages]
    st["free_pages"].copy_(stack)
    # pages for the new tokens, from the top
    new = (j >= old[:, None]) & (j < (old + need)[:, None])
    rank = new.flatten().cumsum(0).view_as(new) - 1
    table.copy_(torch.where(new, stack[(F - 1 - rank).clamp(0, num_pages - 1)], table))
    st["free_count_out"].copy_(F - need.sum())
    t = torch.arange(T, device=lens.device)
    s = torch.searchsorted(st["cu_new"][1:].long(), t, right=True)
    real = s < lens.numel()
    s = s.clamp(max=lens.numel() - 1)
    pos = torch.where(real, lens[s] + t - st["cu_new"].long()[s], 0)
    at = table[s, (pos // page).clamp(max=max_pages - 1)].long() * page + pos % page
    st["slots"].copy_(torch.where(real, at, -1))
    st["positions"].copy_(pos)


def _run_cache(st, case):
    page = case["page"]
    _run_plan(st, case)
    slots, pos = st["slots"].long(), st["positions"]
    real = (slots >= 0)[:, None, None]
    q = _norm_rotate(st["q"], st["wq"], st["cos"], st["sin"], pos, case).to(BF16)
    st["Q"].copy_(torch.where(real, q, st["Q"]))
    k = _norm_rotate(st["k"], st["wk"], st["cos"], st["sin"], pos, case).to(BF16)
    keep = slots >= 0
    at = slots[keep]
    st["K"][at // page, :, at % page] = k[keep]
    st["V"][at // page, :, at % page] = st["v"][keep]
    # a page's mean is renewed by the last of its new tokens
    p = slots // page
    last = keep & (p != torch.cat((p[1:], p.new_full((1,), -2))))
    p, n = p[last], slots[last] % page + 1
    mask = (torch.arange(page, device=p.device) < n[:, None])[:, None, :, None]
    st["ksum"][p] = (torch.where(mask, st["K"][p].float(), 0).sum(2) / n[:, None, None]).to(BF16)
    return _cache_outputs(st)


def _cache_outputs(st):
    return {k: st[k] for k in ("lens_out", "free_count_out", "free_pages", "table", "cu_new", "slots", "positions", "Q", "K", "V", "ksum")}


def _run_select(st, case):
    S, Hq, Hkv, d, page = case["S"], case["Hq"], case["Hkv"], case["d"], case["page"]
    q = st["Q"].float().view(S, Hkv, Hq // Hkv, d)
    kbar = st["ksum"][st["table"].long()].float().permute(0, 2, 3, 1)  # [S, Hkv, d, pages]
    j = torch.arange(st["max_pages"], device=q.device)
    n = (st["lens"].long()[:, None] - j * page).clamp(0, page)[:, None, None]
    x = q @ kbar / math.sqrt(d) + torch.log(n.float())
    e = torch.exp(x - x.amax(-1, keepdim=True))
    p = (e / e.sum(-1, keepdim=True)).mean(2)
    st["P"].copy_(torch.where(n[:, :, 0] > 0, p, st["P"]))
    return {"P": st["P"]}


def _run_topk(st, case):
    page, P = case["page"], st["P"]
    n = (st["lens"].long() + page - 1) // page
    kb = torch.minimum(torch.floor(_keep(case) * n.double() + 0.5).long().clamp(min=1), n)
    j = torch.arange(st["max_pages"], device=P.device)
    forced = (j >= (n - torch.clamp(kb, max=case["recent"]))[:, None]) & (j < n[:, None])
    score = torch.where(forced[:, None], math.inf, P)
    score = torch.where((j < n[:, None])[:, None], score, -1.0)
    order = score.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(P, dtype=torch.bool).scatter(-1, order, (j < kb[:, None])[:, None].expand_as(P))
    idx = torch.where(kept, j, st["max_pages"]).sort(dim=-1).values
    st["idx"].copy_(torch.where((j < kb[:, None])[:, None], idx, st["idx"]))
    st["count"].copy_(kb[:, None].expand_as(st["count"]))


def _run_attend(st, case):
    S, Hq, Hkv, d, page = case["S"], case["Hq"], case["Hkv"], case["d"], case["page"]
    lens = st["lens"].long()
    if case["keep"]:
        _run_topk(st, case)
        j = st["idx"][:, :, :st["most"]].long()
        real = torch.arange(st["most"], device=j.device) < st["count"][:, :, None]
    else:
        j = torch.arange(st["max_pages"], device=lens.device).expand(S, Hkv, -1)
        real = torch.ones_like(j, dtype=torch.bool)
    pages = st["table"].long()[torch.arange(S, device=j.device)[:, None, None], j]
    head = torch.arange(Hkv, device=j.device)[None, :, None]
    key = j[..., None] * page + torch.arange(page, device=j.device)
    mask = (real[..., None] & (key < lens[:, None, None, None])).flatten(2)
    q = st["Q"].float().view(S, Hkv, Hq // Hkv, d) / math.sqrt(d)
    x = q @ st["K"][pages, head].flatten(2, 3).float().transpose(-1, -2)
    x = torch.where(mask[:, :, None], x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = e / e.sum(-1, keepdim=True) @ torch.where(mask[..., None], st["V"][pages, head].flatten(2, 3).float(), 0)
    st["O"].copy_(o.view(S, Hq, d))
    return {"idx": st["idx"], "count": st["count"], "O": st["O"]} if case["keep"] else {"O": st["O"]}


# ------------------------------------------------------ the library's calls
def _own_handles(st, case):
    """What a program makes once and keeps: the parameters, the norm's weights and tables, a workspace."""
    import block_sparse_attention_queries_b200 as ab
    if "cos" in st:
        st["nr"] = ab.NormRope(norm=case["norm"], interleaved=case["interleaved"], eps=EPS, wq=st["wq"], wk=st["wk"], cos=st["cos"],
                               sin=st["sin"])
    if case["kind"] == "rope":
        st["p"] = ab.Params(B=case["B"], H=case["H"], L=case["L"], d=case["d"], L_kv=case["Lk"])
    else:
        st["p"] = ab.PagedParams(S=case["S"], Hq=case["Hq"], Hkv=case["Hkv"], d=case["d"], page=case["page"], num_pages=st["num_pages"],
                                 max_pages=st["max_pages"], keep_ratio=case.get("keep") or 1.0, recent=case.get("recent", 0))
        st["ws"] = ab.alloc_paged_workspace(st["p"], "cuda", select=case["kind"] == "select")
    st["ab"] = ab


def _run_own(st, case):
    if "ab" not in st:
        _own_handles(st, case)
    ab, p, kind = st["ab"], st["p"], case["kind"]
    if kind == "rope":
        Q, K, V = ab.ab_qk_norm_rope(p, st["nr"], st["q"], st["k"], st["v"], pos_q=st["pos_q"], pos_k=st["pos_k"], out=st["out"])
        return {"Q": Q, "K": K, "V": V}
    if kind == "cache":
        ab.ab_paged_plan(p, st["n_new"], st["lens"], st["table"], st["free_pages"], st["free_count"], lens_out=st["lens_out"],
                         free_count_out=st["free_count_out"], out=(st["cu_new"], st["slots"], st["positions"]))
        ab.ab_paged_append(p, st["nr"], st["q"], st["k"], st["v"], st["slots"], st["positions"], st["K"], st["V"], ksum=st["ksum"],
                           out=st["Q"])
        return _cache_outputs(st)
    if kind == "select":
        return {"P": ab.ab_paged_select(p, st["Q"], st["ksum"], st["table"], st["lens"], workspace=st["ws"], out=st["P"])}
    lists = ab.ab_paged_topk(p, st["P"], st["lens"], out=(st["idx"], st["count"])) if case["keep"] else (None, None)
    O = ab.ab_attention_paged(p, st["Q"], st["K"], st["V"], st["table"], st["lens"], idx=lists[0], count=lists[1], workspace=st["ws"],
                              out=st["O"])
    return {"idx": lists[0], "count": lists[1], "O": O} if case["keep"] else {"O": O}


def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    return {"rope": _run_rope, "cache": _run_cache, "select": _run_select, "attend": _run_attend}[case["kind"]](st, case)


# -------------------------------------------------------------------- work
def work(case):
    kind, d = case["kind"], case["d"]
    if kind == "rope":
        vectors = case["B"] * case["H"] * (case["L"] + 2 * case["Lk"])
        rows = (case["L"] if case["L"] == case["Lk"] else case["L"] + case["Lk"]) * (case["B"] if case["pos"] else 1)
        return {"bytes": 4 * d * vectors + 4 * d * rows, "flops": 9 * d * vectors}
    S, Hq, Hkv, page = case["S"], case["Hq"], case["Hkv"], case["page"]
    lens = [n for n, _ in _requests(case)]
    pages = sum(_cdiv(n, page) for n in lens)
    if kind == "cache":
        new = [(n, m) for n, m in _requests(case) if m > 0]
        tokens = sum(m for _, m in new)
        touched = sum(_cdiv(n + m, page) - n // page for n, m in new)
        old = sum(n % page for n, _ in new)  # keys that were in a touched page already
        moved = 4 * d * tokens * (Hq + 2 * Hkv) + 4 * d * tokens
        return {"bytes": moved + 2 * d * Hkv * (touched + old) + 12 * tokens + 16 * S + 4 * touched,
                "flops": 9 * d * tokens * (Hq + Hkv) + d * Hkv * (tokens + old)}
    if kind == "select":
        return {"bytes": pages * (2 * d * Hkv + 4 * Hkv + 4) + 2 * d * S * Hq, "flops": 2 * d * Hq * pages}
    keys = sum(lens)
    if case["keep"]:
        counts = [min(max(int(math.floor(_keep(case) * _cdiv(n, page) + 0.5)), 1), _cdiv(n, page)) for n in lens]
        keys = sum(min(c * page, n) for c, n in zip(counts, lens))
        lists = Hkv * (4 * pages + 4 * sum(counts) + 4 * S)
    else:
        lists = 0
    return {"bytes": 4 * d * Hkv * keys + lists + 4 * pages + 4 * d * S * Hq, "flops": 4 * d * Hq * keys}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "select": _exact_select, "attend": _exact_attend}[case["kind"]](st, case)


def _exact_tokens(x, w, st, pos, case):
    """Tokens x [n, H, d] at positions pos [n]: the rotation as a product of complex numbers."""
    x = x.double()
    if case["norm"] != "none":
        dims = (1, 2) if case["norm"] == "token" else (2,)
        x = x / (x.pow(2).mean(dims, keepdim=True) + EPS).sqrt() * w.double()
    turn = torch.complex(st["cos"].double()[pos.long()], st["sin"].double()[pos.long()])[:, None]
    n, H, d = x.shape
    pairs = x.view(n, H, d // 2, 2) if case["interleaved"] else x.view(n, H, 2, d // 2).transpose(2, 3)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    return y.reshape(n, H, d) if case["interleaved"] else y.transpose(2, 3).reshape(n, H, d)


def _exact_rope(st, case):
    got = {}
    for name, w, pos in (("q", st["wq"], st["pos_q"]), ("k", st["wk"], st["pos_k"])):
        x = st[name]
        parts = []
        for b in range(case["B"]):
            at = torch.arange(x.shape[1], device="cuda") if pos is None else pos[b]
            parts.append(_exact_tokens(x[b], w, st, at, case).permute(1, 0, 2))
        got[name.upper()] = torch.stack(parts)
    got["V"] = st["v"].double().permute(0, 2, 1, 3)
    return got


def _exact_cache(st, case):
    """The lists by hand, request after request; then the new tokens one page at a time."""
    page, T = case["page"], st["T"]
    lens, news, table, free = (st[k].tolist() for k in ("lens", "n_new", "table", "free_pages"))
    top = st["free_count"].item()
    for s, n in enumerate(news):
        if n < 0:
            for j in range(_cdiv(lens[s], page)):
                free[top] = table[s][j]
                top += 1
    cu, slots, positions, after, open_ = [0], [], [], [], True
    for s, n in enumerate(news):
        k = max(n, 0)
        if lens[s] + k > st["max_pages"] * page:
            k = 0
        old = _cdiv(lens[s], page)
        need = _cdiv(lens[s] + k, page) - old if n >= 0 else 0
        open_ = open_ and need <= top and len(slots) + k <= T
        if not open_:
            k = need = 0
        for j in range(need):
            top -= 1
            table[s][old + j] = free[top]
        for i in range(k):
            at = lens[s] + i
            positions.append(at)
            slots.append(table[s][at // page] * page + at % page)
        after.append(0 if n < 0 else lens[s] + k)
        cu.append(len(slots))
    used = len(slots)
    slots += [-1] * (T - used)
    positions += [0] * (T - used)
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    at, pos = whole(slots[:used]).long(), whole(positions[:used])
    Q = st["Q"].double()
    K, V, ksum = (st[k].double() for k in ("K", "V", "ksum"))
    Q[:used] = _exact_tokens(st["q"][:used], st["wq"], st, pos, case)
    K[at // page, :, at % page] = _exact_tokens(st["k"][:used], st["wk"], st, pos, case)
    V[at // page, :, at % page] = st["v"][:used].double()
    fill = {}
    for x in slots[:used]:
        fill[x // page] = max(fill.get(x // page, 0), x % page + 1)
    for n in sorted(set(fill.values())):
        p = whole([k for k, v in fill.items() if v == n]).long()
        ksum[p] = K[p, :, :n].to(BF16).double().mean(2)
    return {"lens_out": whole(after), "free_count_out": whole([top]), "free_pages": whole(free), "table": whole(table), "cu_new": whole(cu),
            "slots": whole(slots), "positions": whole(positions), "Q": Q, "K": K, "V": V, "ksum": ksum}


def _exact_select(st, case):
    page, G = case["page"], case["Hq"] // case["Hkv"]
    P = torch.zeros_like(st["P"], dtype=torch.float64)
    for s, n in enumerate(st["lens"].tolist()):
        k = _cdiv(n, page)
        kbar = st["ksum"][st["table"][s, :k].long()].double()
        size = torch.full((k,), page, dtype=torch.float64, device="cuda")
        size[-1] = n - (k - 1) * page
        for h in range(case["Hq"]):
            x = kbar[:, h // G] @ st["Q"][s, h].double() / math.sqrt(case["d"]) + size.log()
            P[s, h // G, :k] += torch.softmax(x, 0) / G
    return {"P": P}


def _exact_attend(st, case):
    page, Hkv, d = case["page"], case["Hkv"], case["d"]
    G = case["Hq"] // Hkv
    O = torch.zeros_like(st["O"], dtype=torch.float64)
    lists = {}
    if case["keep"]:
        lists = {"idx": st["idx"].clone(), "count": st["count"].clone()}
    for s, n in enumerate(st["lens"].tolist()):
        k = _cdiv(n, page)
        for g in range(Hkv):
            j = torch.arange(k, device="cuda")
            if case["keep"]:
                kb = min(max(int(math.floor(_keep(case) * k + 0.5)), 1), k)
                recent = min(case["recent"], kb)
                by = torch.argsort(st["P"][s, g, :k - recent], descending=True, stable=True)[:kb - recent]
                j = torch.cat((by.sort().values, j[k - recent:]))
                lists["idx"][s, g, :kb], lists["count"][s, g] = j.int(), kb
            p = st["table"][s].long()[j]
            real = (j[:, None] * page + torch.arange(page, device="cuda") < n).flatten()
            keys = st["K"][p, g].reshape(-1, d)[real].double()
            values = st["V"][p, g].reshape(-1, d)[real].double()
            x = st["Q"][s, g * G:(g + 1) * G].double() @ keys.T / math.sqrt(d)
            O[s, g * G:(g + 1) * G] = torch.softmax(x, -1) @ values
    return {**lists, "O": O}
