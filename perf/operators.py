"""The cache operators' cases: what they are given, their plain form in elementary
torch operations, and their definition in 64 bits.

Four operators around a key/value cache that a block layout routes:

* ``weights``: the attention weight that every key of a prompt has received,
  w[u] = sum over the query heads of its group and the tokens t that may read
  it of exp(scale <q_t, k_u> - lse_t);
* ``step``: one decode step over the paged cache that also adds the step's
  weights to the running ones;
* ``evict``: every key/value head keeps its `budget` cached tokens of largest
  accumulated weight (the `recent` newest always), the kept ones moved into
  the first slots;
* ``tree``: attention of a tree of drafted tokens over the paged cache and
  their own ancestors.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a 32K prompt on the dyadic route (16 query on 8 key/value heads): its weights, before the cache is cut
        {"name": "weights_dyadic_32k", "op": "weights", "batch": 1, "H": 16, "G": 8, "n": 32768, "d": 128, "B": 64,
         "route": "dyadic", "L": 1, "density": 0.0},
        # a ragged prompt on the band route with one key/value head for each query head
        {"name": "weights_band_9001", "op": "weights", "batch": 1, "H": 32, "G": 32, "n": 9001, "d": 128, "B": 128,
         "route": "band", "L": 1, "density": 0.0},
        # two short prompts of small heads, every head on a random route of its own
        {"name": "weights_random_2500", "op": "weights", "batch": 2, "H": 8, "G": 4, "n": 2500, "d": 64, "B": 64,
         "route": "random", "L": 8, "density": 0.3},
        # one token of one user at the end of a 32K context: the smallest step, where latency counts
        {"name": "step_dyadic_b1", "op": "step", "batch": 1, "H": 16, "G": 8, "n": 32768, "d": 128, "B": 64,
         "route": "dyadic", "L": 1, "density": 0.0},
        # sixteen users whose every token reads the whole cache, as a cache that evicts is read
        {"name": "step_full_b16_16k", "op": "step", "batch": 16, "H": 16, "G": 8, "n": 16384, "d": 128, "B": 64,
         "route": "full", "L": 1, "density": 0.0},
        # two long contexts on random routes, one for each head
        {"name": "step_random_131k", "op": "step", "batch": 2, "H": 8, "G": 8, "n": 131072, "d": 128, "B": 128,
         "route": "random", "L": 8, "density": 0.1},
        # the cut after long prompts: a quarter of the tokens stays
        {"name": "evict_prompt_32k", "op": "evict", "batch": 2, "H": 8, "G": 8, "n": 32768, "d": 128, "B": 64,
         "budget": 8192, "recent": 1024, "over": 0, "ids": False},
        # the cut that a batch makes each time it has filled one page over its budget
        {"name": "evict_page_b32", "op": "evict", "batch": 32, "H": 8, "G": 8, "n": 4224, "d": 128, "B": 64,
         "budget": 4096, "recent": 512, "over": 64, "ids": True},
        # a small cache of odd sizes, cut before, so its slots are out of order
        {"name": "evict_odd_d64", "op": "evict", "batch": 5, "H": 2, "G": 2, "n": 1000, "d": 64, "B": 128,
         "budget": 333, "recent": 50, "over": 0, "ids": True},
        # one user's drafted tree on the dyadic route
        {"name": "tree_dyadic_b1", "op": "tree", "batch": 1, "H": 16, "G": 8, "n": 32768, "d": 128, "B": 64,
         "route": "dyadic", "L": 1, "density": 0.0, "T": 26, "chain": 0.3},
        # eight users' full trees over whole caches
        {"name": "tree_full_b8_16k", "op": "tree", "batch": 8, "H": 16, "G": 8, "n": 16384, "d": 128, "B": 64,
         "route": "full", "L": 1, "density": 0.0, "T": 64, "chain": 0.3},
        # short drafted chains over long contexts, a random route for each head
        {"name": "tree_chain_131k", "op": "tree", "batch": 2, "H": 8, "G": 8, "n": 131072, "d": 128, "B": 128,
         "route": "random", "L": 8, "density": 0.1, "T": 5, "chain": 1.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["weights", "step", "evict", "tree"])
    d, B = rng.choice([64, 128]), rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 8])
    case = {"op": op, "G": G, "d": d, "B": B}
    if op == "evict":
        n = _log(rng, 200, 32768)
        budget = max(1, min(n, int(n * rng.uniform(0.1, 1.0))))
        over = rng.choice([0, 0, 1, B, _log(rng, 1, 2 * B)])
        case.update(H=G, n=n, batch=_log(rng, 1, max(1, min(32, 65536 // n))), budget=budget,
                    recent=int(budget * rng.uniform(0.0, 0.5)), over=over if budget + over <= n else 0,
                    ids=rng.random() < 0.5)
        return case
    route = rng.choice(["dyadic", "band", "random", "full"])
    H = G * rng.choice([1, 2, 2, 3, 4]) if G < 8 else G * rng.choice([1, 2])
    L = rng.choice([1, H]) if route == "random" else 1
    most = {"weights": {"full": 4096, "random": 8192}.get(route, 16384),
            "step": {"full": 16384}.get(route, 65536), "tree": {"full": 16384}.get(route, 65536)}[op]
    n = _log(rng, 300, most)
    case.update(H=H, n=n, route=route, L=L, density=round(rng.uniform(0.05, 0.3), 3) if route == "random" else 0.0)
    if op == "weights":
        case["batch"] = _log(rng, 1, max(1, min(4, 16384 // n)))
    else:
        case["batch"] = _log(rng, 1, max(1, min(16, 131072 // n)))
    if op == "tree":
        case.update(T=_log(rng, 1, 128 if case["batch"] * n <= 65536 else 64), chain=rng.choice([0.0, 0.3, 0.7, 1.0]))
    return case


# ------------------------------------------------------------------ what a program has in hand

def _kept(case):
    """Kept key blocks of every query block, truth values [L][nb][nb]."""
    nb = -(-case["n"] // case["B"])
    i, j = np.arange(nb)[:, None], np.arange(nb)[None, :]
    if case["route"] == "full":
        m = (j <= i)[None]
    elif case["route"] == "band":
        m = ((j <= i) & ((i - j <= 2) | (j == 0)))[None]
    elif case["route"] == "dyadic":
        gap = i - j
        m = ((gap >= 0) & ((gap <= 2) | (j == 0) | ((gap >= 4) & ((gap & (gap - 1)) == 0))))[None]
    else:
        r = np.random.default_rng(17)
        m = (r.random((case["L"], nb, nb)) < case["density"]) | (i == j) | (j == 0)
        m &= j <= i
    return np.ascontiguousarray(m)


def _layout(case):
    """The framework's layout of the same route, which a program builds once."""
    import block_sparse_long_bsa_b200 as bsa
    n, B, dev = case["n"], case["B"], torch.cuda.current_device()
    route = case.get("route", "full")
    if route == "full":
        return bsa.Layout(bsa.PATTERN_BAND_GLOBAL, n, B, 1, dev, window=-(-n // B), global_first=0)
    if route == "band":
        return bsa.Layout(bsa.PATTERN_BAND_GLOBAL, n, B, 1, dev, window=2, global_first=1)
    if route == "dyadic":
        return bsa.Layout(bsa.PATTERN_DYADIC, n, B, 1, dev, window=2, global_first=1, dyadic_kmin=2)
    return bsa.Layout(bsa.PATTERN_EXPLICIT, n, B, case["L"], dev, mask=_kept(case).astype(np.uint8))


def _rows(case):
    """Each query block's kept key blocks in ascending order: [L][nb][R] and which of them are meant."""
    m = torch.from_numpy(_kept(case)).cuda()
    count = m.sum(-1)
    r = int(count.max())
    idx = torch.sort((~m).to(torch.uint8), dim=-1, stable=True).indices[..., :r].contiguous()
    return idx, torch.arange(r, device="cuda") < count[..., None]


def _ends(case):
    """Cached tokens of each sequence: the last one full, the others up to a quarter shorter."""
    room = case.get("T", 0)
    full = max(1, case["n"] - room)
    return [max(1, full - (case["batch"] - 1 - b) * (full // 4) // max(1, case["batch"])) for b in range(case["batch"])]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _cache(case, g):
    nb = -(-case["n"] // case["B"])
    pages = case["batch"] * nb
    kc = _normal(g, pages, case["G"], case["B"], case["d"])
    vc = _normal(g, pages, case["G"], case["B"], case["d"])
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(case["batch"], nb)
    return kc, vc, table


def _inputs(case, seed):
    g = _gen(seed)
    b, H, G, n, d = case["batch"], case["H"], case["G"], case["n"], case["d"]
    s = {"case": case, "scale": d ** -0.5}
    if case["op"] == "weights":
        s["q"], s["k"] = _normal(g, b * H, n, d), _normal(g, b * G, n, d)
        s["weights"] = torch.zeros((b * G, n), device="cuda")
        return s
    s["k_cache"], s["v_cache"], s["table"] = _cache(case, g)
    if case["op"] == "step":
        s["q"] = _normal(g, b * H, d)
        s["positions"] = torch.tensor(_ends(case), dtype=torch.int32, device="cuda") - 1
        s["weights"] = torch.rand((b * G, n), generator=g, device="cuda") * 4
        s["o"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros(b * H, device="cuda")
    elif case["op"] == "evict":
        ends = [case["budget"] + case["over"]] * b if case["over"] else _ends(case)
        s["lengths"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        # few tokens hold most of the weight; many of the rest have none at all, so that ties are met
        w = torch.exp(2 * torch.randn((b * G, n), generator=g, device="cuda"))
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.2, 0.0, w)
        if case["ids"]:
            # what an earlier cut leaves: each head's slots hold tokens in an order of their own, of a longer sequence
            order = torch.rand(w.shape, generator=g, device="cuda").argsort(-1)
            s["tokens"] = (2 * order + torch.randint(0, 2, w.shape, generator=g, device="cuda")).to(torch.int32)
        else:
            s["tokens"] = None
        s["weights_out"] = torch.zeros_like(w)
        s["tokens_out"] = torch.zeros(w.shape, dtype=torch.int32, device="cuda")
        s["lengths_out"] = torch.zeros(b, dtype=torch.int32, device="cuda")
    else:
        T = case["T"]
        s["q"] = _normal(g, b * H, T, d)
        s["k_tree"], s["v_tree"] = _normal(g, b * G, T, d), _normal(g, b * G, T, d)
        s["lengths"] = torch.tensor(_ends(case), dtype=torch.int32, device="cuda")
        # a token follows the one before it (a chain), or any earlier one near the root, or the context itself (-1)
        i = torch.arange(T, device="cuda")
        u = torch.rand((b, T), generator=g, device="cuda")
        other = torch.floor(u * u * (i + 1)).to(torch.int64) - 1
        chain = torch.rand((b, T), generator=g, device="cuda") < case["chain"]
        par = torch.where(chain, i - 1, other.clamp(max=T)).clamp(min=-1)
        # the last sequences of a batch have drafted fewer tokens: the rows behind are unused (-2)
        used = torch.tensor([T if x == 0 else max(1, T - x) for x in range(b)], device="cuda")
        s["parents"] = torch.where(i[None] < used[:, None], torch.minimum(par, i - 1), -2).to(torch.int32)
        s["o"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((b * H, T), device="cuda")
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] != "evict":
        s["rows"], s["valid"] = _rows(case)
    if case["op"] == "weights":
        s["lse"] = _prompt_lse(s)
    if own:
        import block_sparse_long_bsa_b200 as bsa
        s["layout"] = _layout(case)
        b, H, G, n, d = case["batch"], case["H"], case["G"], case["n"], case["d"]
        h = s["layout"].handle
        need = {"weights": lambda: bsa.bsa_attention_weights_workspace_bytes(h, b * H, b * G),
                "step": lambda: bsa.bsa_decode_weights_workspace_bytes(h, b, b * H, b * G, d),
                "evict": lambda: bsa.bsa_evict_workspace_bytes(h, b, b * G, case.get("budget", 1)),
                "tree": lambda: bsa.bsa_decode_tree_workspace_bytes(h, b, b * H, b * G, case.get("T", 1), d)}[case["op"]]()
        s["workspace"] = torch.empty(max(16, need), dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"weights": _own_weights, "step": _own_step, "evict": _own_evict, "tree": _own_tree}[op](s)
    return {"weights": _plain_weights, "step": _plain_step, "evict": _plain_evict, "tree": _plain_tree}[op](s)


def _own_weights(s):
    import block_sparse_long_bsa_b200 as bsa
    s["weights"].zero_()
    return bsa.attention_weights(s["q"], s["k"], s["lse"], s["layout"], s["weights"], s["scale"],
                                 workspace=s["workspace"])


def _own_step(s):
    import block_sparse_long_bsa_b200 as bsa
    o, lse = bsa.decode_weights(s["q"], s["k_cache"], s["v_cache"], s["table"], s["positions"], s["layout"],
                                s["case"]["batch"], s["weights"], s["scale"], o=s["o"], lse=s["lse"],
                                workspace=s["workspace"])
    return {"o": o, "lse": lse, "weights": s["weights"]}


def _own_evict(s):
    import block_sparse_long_bsa_b200 as bsa
    w, t, n = bsa.evict(s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["weights"], s["layout"],
                        s["case"]["budget"], s["case"]["recent"], tokens=s["tokens"], weights_out=s["weights_out"],
                        tokens_out=s["tokens_out"], lengths_out=s["lengths_out"], workspace=s["workspace"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": w, "tokens": t, "lengths": n}


def _own_tree(s):
    import block_sparse_long_bsa_b200 as bsa
    o, lse = bsa.decode_tree(s["q"], s["k_tree"], s["v_tree"], s["k_cache"], s["v_cache"], s["table"], s["lengths"],
                             s["parents"], s["layout"], s["scale"], o=s["o"], lse=s["lse"],
                             workspace=s["workspace"])
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ the plain forms

def _heads(case):
    """For each folded query head: its sequence, its key/value head of the batch, its layout head."""
    f = torch.arange(case["batch"] * case["H"], device="cuda")
    return f // case["H"], f // (case["H"] // case["G"]), f % case["L"]


def _pad(x, n):
    return torch.cat([x, x.new_zeros((x.shape[0], n - x.shape[1]) + x.shape[2:])], 1) if n > x.shape[1] else x


def _prompt_scores(s):
    """scale <q, k> of every token with the keys of its block's kept blocks [heads][nb][B][R*B], which may be read,
    and their tokens."""
    case = s["case"]
    n, B, d = case["n"], case["B"], case["d"]
    nb = -(-n // B)
    _, kv, lay = _heads(case)
    q = _pad(s["q"].float(), nb * B).view(-1, nb, B, d)
    k = _pad(s["k"].float(), nb * B).view(-1, nb, B, d)
    rows, valid = s["rows"][lay], s["valid"][lay]                    # [heads][nb][R]
    kept = k[kv[:, None, None], rows].flatten(2, 3)                  # [heads][nb][R*B][d]
    scores = s["scale"] * (q @ kept.transpose(-1, -2))
    key = (rows[..., None] * B + torch.arange(B, device="cuda")).flatten(2, 3)
    tok = torch.arange(nb * B, device="cuda").view(nb, B)
    may = valid.repeat_interleave(B, -1)[:, :, None] & (key[:, :, None] <= tok[..., None]) & (tok[..., None] < n)
    return scores, may, key


def _log_sum(x):
    """log of the sum of exp over the last axis; -inf where all are -inf."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == NEG, torch.zeros_like(top), top)
    return (torch.exp(x - top).sum(-1, keepdim=True).log() + top).squeeze(-1)


def _prompt_lse(s):
    scores, may, _ = _prompt_scores(s)
    return _log_sum(torch.where(may, scores, NEG)).flatten(1, 2)[:, : s["case"]["n"]].contiguous()


def _plain_weights(s):
    case = s["case"]
    n, B = case["n"], case["B"]
    nb = -(-n // B)
    scores, may, key = _prompt_scores(s)
    lse = _pad(s["lse"], nb * B).view(-1, nb, B, 1)
    p = torch.where(may, torch.exp(scores - lse), 0.0).sum(2)         # [heads][nb][R*B]
    at = _heads(case)[1][:, None, None] * (nb * B) + key
    total = torch.zeros(case["batch"] * case["G"] * nb * B, dtype=torch.float64, device="cuda")
    total.index_add_(0, at.flatten(), p.double().flatten())
    s["weights"].zero_()
    s["weights"] += total.view(-1, nb * B)[:, :n].float()
    return s["weights"]


def _plain_step(s):
    case = s["case"]
    B, G = case["B"], case["G"]
    seq, kv, lay = _heads(case)
    pos = s["positions"].long()[seq]
    rows, valid = s["rows"][lay, pos // B], s["valid"][lay, pos // B]  # [heads][R]
    page = s["table"].long()[seq[:, None], rows]
    keys = s["k_cache"][page, (kv % G)[:, None]].flatten(1, 2).float()
    vals = s["v_cache"][page, (kv % G)[:, None]].flatten(1, 2).float()
    key = (rows[..., None] * B + torch.arange(B, device="cuda")).flatten(1)
    may = valid.repeat_interleave(B, -1) & (key <= pos[:, None])
    x = torch.where(may, s["scale"] * (keys @ s["q"].float()[..., None]).squeeze(-1), NEG)
    lse = _log_sum(x)
    p = torch.where(may, torch.exp(x - lse[:, None]), 0.0)
    s["o"].copy_((p[:, None] @ vals).squeeze(1).to(torch.bfloat16))
    s["lse"].copy_(lse)
    add = torch.zeros_like(s["weights"], dtype=torch.float64)
    add.view(-1).index_add_(0, (kv[:, None] * case["n"] + key)[may], p[may].double())
    s["weights"] += add.float()
    return {"o": s["o"], "lse": s["lse"], "weights": s["weights"]}


def _plain_evict(s):
    case = s["case"]
    b, G, n, B, budget = case["batch"], case["G"], case["n"], case["B"], case["budget"]
    slot = torch.arange(n, device="cuda").expand(b * G, n)
    length = s["lengths"].long().repeat_interleave(G)[:, None]
    used = slot < length
    ids = slot if s["tokens"] is None else s["tokens"].long()
    newest = torch.where(used, ids, -1).amax(1, keepdim=True)
    kept = torch.minimum(length, torch.full_like(length, budget))
    # the newest first, then by weight (NaN behind all), the lower slot at a tie, unused slots last
    w = torch.where(torch.isnan(s["weights"]), NEG, s["weights"])
    by_weight = torch.sort(w, dim=1, descending=True, stable=True).indices
    rank = torch.where(used, torch.where(ids > newest - case["recent"], 0, 1), 2).gather(1, by_weight)
    order = by_weight.gather(1, torch.sort(rank, dim=1, stable=True).indices)
    stays = torch.zeros((b * G, n), dtype=torch.bool, device="cuda").scatter_(1, order, slot < kept)
    hole, mover = (slot < kept) & ~stays, (slot >= kept) & stays
    row = torch.arange(b * G, device="cuda")[:, None].expand(b * G, n)
    # the holes of a row and its movers are as many: the i-th hole takes the i-th mover
    src = slot.clone()
    src[hole] = slot[mover]
    r, dst, frm = row[hole], slot[hole], src[hole]
    table = s["table"].long()
    to, at = table[r // G, dst // B], table[r // G, frm // B]
    s["k_cache"][to, r % G, dst % B] = s["k_cache"][at, r % G, frm % B]
    s["v_cache"][to, r % G, dst % B] = s["v_cache"][at, r % G, frm % B]
    s["weights_out"].copy_(torch.where(slot < kept, s["weights"].gather(1, src), 0.0))
    s["tokens_out"].copy_(torch.where(slot < kept, ids.gather(1, src), newest + 1 + slot - kept).to(torch.int32))
    s["lengths_out"].copy_(kept.view(b, G)[:, 0])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "weights": s["weights_out"], "tokens": s["tokens_out"],
            "lengths": s["lengths_out"]}


def _plain_tree(s):
    case = s["case"]
    B, G, T = case["B"], case["G"], case["T"]
    nb = -(-case["n"] // B)
    seq, kv, lay = _heads(case)
    par = s["parents"].long()
    one = torch.arange(T, device="cuda")
    up = (par[..., None] == one).double()                             # [batch][T][T]: is the parent
    above = torch.linalg.matrix_power(up + torch.eye(T, device="cuda", dtype=torch.float64), T) > 0
    depth = above.sum(-1) - 1
    length = s["lengths"].long()
    pos = length[:, None] + depth                                     # [batch][T]
    # the block rows that the tree's positions fall in, and the cached keys that each of them keeps
    groups = (T + B - 2) // B + 1
    row = (length // B)[:, None] + torch.arange(groups, device="cuda")
    rows = s["rows"][lay[:, None], row.clamp(max=nb - 1)[seq]]        # [heads][groups][R]
    valid = s["valid"][lay[:, None], row.clamp(max=nb - 1)[seq]]
    page = s["table"].long()[seq[:, None, None], rows]
    keys = s["k_cache"][page, (kv % G)[:, None, None]].flatten(1, 3).float()
    vals = s["v_cache"][page, (kv % G)[:, None, None]].flatten(1, 3).float()
    key = (rows[..., None] * B + torch.arange(B, device="cuda")).flatten(2)
    in_row = (pos // B)[:, None] == row[..., None]                    # [batch][groups][T]
    cached = valid.repeat_interleave(B, -1) & (key < length[seq][:, None, None])
    may = in_row[seq][..., None] & cached[:, :, None]                 # [heads][groups][T][R*B]
    may = may.transpose(1, 2).flatten(2)
    q = s["q"].float()
    x = torch.where(may, s["scale"] * (q @ keys.transpose(-1, -2)), NEG)
    # an ancestor is read where the token's row keeps the ancestor's block
    blk = (pos // B).clamp(max=nb - 1)[seq]
    in_list = (s["rows"][lay[:, None], blk][:, :, None] == blk[:, None, :, None]) & s["valid"][lay[:, None], blk][:, :, None]
    mine = above[seq] & in_list.any(-1)
    y = torch.where(mine, s["scale"] * (q @ s["k_tree"].float()[kv].transpose(-1, -2)), NEG)
    both, allowed = torch.cat([x, y], -1), torch.cat([may, mine], -1)
    lse = _log_sum(both)
    p = torch.where(allowed, torch.exp(both - lse[..., None]), 0.0)
    o = p @ torch.cat([vals, s["v_tree"].float()[kv]], 1)
    used = (par >= -1)[seq]
    s["o"].copy_(torch.where(used[..., None], o.to(torch.bfloat16), s["o"]))
    s["lse"].copy_(torch.where(used, lse, s["lse"]))
    return {"o": s["o"], "lse": s["lse"]}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "weights":
        s["rows"], s["valid"] = _rows(case)
        s["lse"] = _prompt_lse(s)
    return {"weights": _exact_weights, "step": _exact_step, "evict": _exact_evict, "tree": _exact_tree}[case["op"]](s)


def _exact_weights(s):
    """Column by column: a key block and all the tokens whose blocks keep it."""
    case = s["case"]
    n, B, g = case["n"], case["B"], case["H"] // case["G"]
    nb = -(-n // B)
    m = _kept(case)
    out = torch.zeros((case["batch"] * case["G"], n), dtype=torch.float64, device="cuda")
    for j in range(nb):
        u = torch.arange(j * B, min(n, (j + 1) * B), device="cuda")
        for lay in range(case["L"]):
            blocks = np.nonzero(m[lay, :, j])[0]
            if not len(blocks):
                continue
            t = (torch.from_numpy(blocks).cuda()[:, None] * B + torch.arange(B, device="cuda")).flatten()
            t = t[t < n]
            f = torch.arange(lay, case["batch"] * case["H"], case["L"], device="cuda")
            x = s["q"][f][:, t].double() @ s["k"][f // g][:, u].double().transpose(1, 2) * s["scale"]
            x -= s["lse"][f][:, t].double()[..., None]
            x = torch.where(u[None] <= t[:, None], x, NEG).exp().sum(1)
            out[:, j * B:j * B + len(u)].index_add_(0, f // g, x)
    return out


def _read(s, b, blocks, end):
    """Keys and values [G][tokens][d] of sequence b's cached tokens below `end` in the given blocks, in 64 bits, and the tokens."""
    B = s["case"]["B"]
    page = s["table"][b].long()[blocks]
    tok = (blocks[:, None] * B + torch.arange(B, device="cuda")).flatten()
    k = s["k_cache"][page].transpose(0, 1).flatten(1, 2)[:, tok < end].double()
    v = s["v_cache"][page].transpose(0, 1).flatten(1, 2)[:, tok < end].double()
    return k, v, tok[tok < end]


def _exact_step(s):
    case = s["case"]
    B, H, G = case["B"], case["H"], case["G"]
    m = _kept(case)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((len(o),), NEG, dtype=torch.float64, device="cuda")
    w = s["weights"].double()
    for b, t in enumerate(s["positions"].tolist()):
        for h in range(H):
            f, kv = b * H + h, h // (H // G)
            if h == 0 or case["L"] > 1:
                k, v, tok = _read(s, b, torch.from_numpy(np.nonzero(m[f % case["L"], t // B])[0]).cuda(), t + 1)
            x = k[kv] @ s["q"][f].double() * s["scale"]
            lse[f] = torch.logsumexp(x, 0)
            p = torch.softmax(x, 0)
            o[f] = p @ v[kv]
            w[b * G + kv, tok] += p
    return {"o": o, "lse": lse, "weights": w}


def _exact_evict(s):
    case = s["case"]
    G, n, B, budget = case["G"], case["n"], case["B"], case["budget"]
    kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    weights = s["weights"].cpu().numpy()
    ids = np.broadcast_to(np.arange(n), weights.shape) if s["tokens"] is None else s["tokens"].cpu().numpy().astype(np.int64)
    table, lengths = s["table"].cpu().numpy(), s["lengths"].tolist()
    w_out, t_out = np.zeros(weights.shape), np.zeros(weights.shape, np.int64)
    for r in range(case["batch"] * G):
        b, length = r // G, lengths[r // G]
        keep = min(length, budget)
        new = ids[r, :length].max() if length else -1
        old = ids[r, :length] <= new - case["recent"]
        chosen = np.lexsort((np.arange(length), -weights[r, :length].astype(np.float64), old))[:keep]
        low = set(chosen[chosen < keep].tolist())
        holes = np.array([x for x in range(keep) if x not in low], dtype=np.int64)
        movers = np.sort(chosen[chosen >= keep])
        src = np.arange(keep)
        src[holes] = movers
        w_out[r, :keep], t_out[r, :keep] = weights[r, src], ids[r, src]
        t_out[r, keep:] = new + 1 + np.arange(n - keep)
        to, at = (torch.from_numpy(x).cuda() for x in (holes, movers))
        page = torch.from_numpy(table[b].astype(np.int64)).cuda()
        for c in (kc, vc):
            c[page[to // B], r % G, to % B] = c[page[at // B], r % G, at % B]
    return {"k_cache": kc.double(), "v_cache": vc.double(), "weights": torch.from_numpy(w_out),
            "tokens": torch.from_numpy(t_out), "lengths": torch.tensor([min(x, budget) for x in lengths])}


def _exact_tree(s):
    """Token by token: the cached keys that its block keeps, then the path from the root down to it."""
    case = s["case"]
    B, H, G, T, L = case["B"], case["H"], case["G"], case["T"], case["L"]
    g = H // G
    m = _kept(case)
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, (length, parents) in enumerate(zip(s["lengths"].tolist(), s["parents"].tolist())):
        have = {}
        for i in range(T):
            if parents[i] == -2:
                continue
            path = [i]
            while parents[path[0]] >= 0:
                path.insert(0, parents[path[0]])
            blk = (length + len(path) - 1) // B
            for lay in range(L):
                if (lay, blk) not in have:
                    have[lay, blk] = _read(s, b, torch.from_numpy(np.nonzero(m[lay, blk])[0]).cuda(), length)
                k, v, _ = have[lay, blk]
                mine = [x for z, x in enumerate(path) if m[lay, blk, (length + z) // B]]
                for h in (range(lay, H, L) if L > 1 else range(0, H, g)):
                    kv, f = h // g, [b * H + h] if L > 1 else list(range(b * H + h, b * H + h + g))
                    q = s["q"][f, i].double()
                    x = torch.cat([q @ k[kv].T, q @ s["k_tree"][b * G + kv, mine].double().T], 1) * s["scale"]
                    lse[f, i] = torch.logsumexp(x, 1)
                    p = torch.softmax(x, 1)
                    c = k.shape[1]
                    o[f, i] = p[:, :c] @ v[kv] + p[:, c:] @ s["v_tree"][b * G + kv, mine].double()
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------ what one pass cannot do without

def work(case):
    b, H, G, n, d, B = (case[x] for x in ("batch", "H", "G", "n", "d", "B"))
    if case["op"] == "evict":
        ends = [case["budget"] + case["over"]] * b if case["over"] else _ends(case)
        moved = 0.0
        for x in ends:
            # of the slots past the budget, as many survive as chance leaves there
            past = max(0, x - case["budget"])
            moved += past * min(x, case["budget"]) / max(1, x)
        read = sum(ends) * G * (8 if case["ids"] else 4)
        return {"bytes": read + b * G * n * 8 + moved * G * 2 * d * 2 * 2, "flops": 0}
    m = _kept(case).astype(np.float64)
    nb = m.shape[1]
    toks = np.minimum(B, n - np.arange(nb) * B).astype(np.float64)
    if case["op"] == "weights":
        pairs = np.einsum("lij,i,j->l", m, toks, toks)
        pairs -= np.einsum("lii,i->l", m, toks * (toks - 1) / 2)
        return {"bytes": (H + G) * b * n * d * 2 + b * n * (4 * H + 8 * G), "flops": 2 * d * float(pairs.mean()) * b * H}
    T = case.get("T", 1)
    keys = union = 0.0
    for e in _ends(case):
        rows = range((e if "T" in case else e - 1) // B, min(nb - 1, (e + T - 1) // B) + 1) if "T" in case else [(e - 1) // B]
        have = np.minimum(B, np.maximum(0, e - np.arange(nb) * B))
        keys += float((m[:, rows[0]] * have).sum(1).mean())
        # what each key/value head has to read: the blocks that any of its query heads keeps
        of = [[f % case["L"] for f in range(kv * (H // G), (kv + 1) * (H // G))] for kv in range(G)]
        union += sum(float((m[x].max(0)[rows[0]] * have).sum()) for x in of)
    small = b * H * T * (4 * d + 4) + (b * G * T * 4 * d if "T" in case else 0)
    return {"bytes": union * 4 * d + small + (union * 8 if case["op"] == "step" else 0),
            "flops": 4.0 * d * H * T * keys}
