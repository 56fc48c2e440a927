"""GPU: the full-attention layer as a decode step uses it, its operators one after another (projections, rotary
positions, cache write, attention, output projection), beside a GDN layer on the same draft, over rounds of
verify and commit.

Each stage is held to its own bar on the values the stage before it stored, so that no bar has to count a
rounding twice: projections 1e-5 beyond their bf16 rounding; rotated q as in the rotary tests (6.1e-7 of |x_a| +
|x_b|, then half a bf16 step); attention as in its own tests, on what gdn_kv_read gives back in fp32."""

import numpy as np
import pytest

from gated_deltanet_linear_verify_amd import workloads as W
from oracle import block
from tests import attn_ref as ref
from tests.gpu_util import half_ulp_bf16, say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HIDDEN, N_Q, N_KV, D, PAGE, ROT, THETA = 256, 8, 2, 128, 16, 64, 1e6
B, T = 3, 9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from gated_deltanet_linear_verify_amd import gdn
    gdn.lib()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _f64(t):
    return t.double().cpu().numpy()


def _beyond_rounding(got, want):
    return float(np.max(np.maximum(np.abs(got - want) - half_ulp_bf16(want), 0.0)) / np.max(np.abs(want)))


class Layer:
    """One layer, its pool (all but the prefix's pages dealt to the entries) and a history in the cache."""

    def __init__(self, fmt, start, prefix=0, seed=0):
        from gated_deltanet_linear_verify_amd import device, gdn
        self.gdn, self.device = gdn, device
        rng = self.rng = np.random.default_rng(seed)
        self.start, self.prefix = np.array(start, np.int32), prefix
        wide = -(-(max(start) + 4 * T) // PAGE)
        shared = -(-prefix // PAGE)
        pages = rng.permutation(B * wide + shared + 1).astype(np.int32)
        self.table = _i32(pages[shared:shared + B * wide].reshape(B, wide))
        self.pages = _i32(pages[:shared]) if prefix else None
        self.plen = _i32([prefix]) if prefix else None
        self.rope = gdn.gdn_rope_init(ROT, theta=THETA)
        self.inp = W.make_attention_inputs(B, T, HIDDEN, N_Q, N_KV, D, seed)
        self.d = device.upload_attention(self.inp, self.rope, fmt=fmt, page_size=PAGE, n_pages=len(pages), prefix=prefix > 0)
        self.kv = self.d["kv"]
        n = int(max(start))  # the history: rows already rotated, in whatever the cache makes of them
        if n:
            rows = torch.from_numpy(rng.standard_normal((B * n, 2 * N_KV, D))).float().cuda()
            gdn.gdn_kv_write(self.kv, rows[:, :N_KV], rows[:, N_KV:], self.table, _i32(np.zeros(B)), _i32(start), B, n)
        if prefix:
            rows = torch.from_numpy(rng.standard_normal((prefix, 2 * N_KV, D))).float().cuda()
            gdn.gdn_kv_write(self.kv, rows[:, :N_KV], rows[:, N_KV:], self.pages[None].contiguous(), _i32([0]), None, 1, prefix)

    def positions(self, start, parent=None):
        depth = np.stack([np.arange(T) if parent is None else W.tree_depths(parent[b]) for b in range(B)])
        return _i32((self.prefix + start[:, None] + depth).reshape(1, B * T))

    def step(self, start, parent=None, n_new=None, stream=None):
        i = lambda a: None if a is None else a if torch.is_tensor(a) else _i32(a)  # noqa: E731
        self.device.attention_step(self.d, self.table, i(start), self.positions(np.asarray(start), parent), i(n_new), i(parent),
                                   self.pages, self.plen, stream)

    def read(self, table, lo, n):
        """k and v [n][N_KV][D] fp64 of one run of pages, as the cache holds them."""
        k, v = (torch.zeros((n, N_KV, D), device="cuda") for _ in range(2))
        if n:
            self.gdn.gdn_kv_read(self.kv, table[None].contiguous(), _i32([lo]), None, k, v, 1, n)
        return _f64(k), _f64(v)


def _draft(seed):
    rng = np.random.default_rng(seed)
    parent = np.stack([W.random_tree(rng, T) for _ in range(B)])
    return parent, [W.tree_path(parent[b], W.tree_accept(rng, parent[b])) for b in range(B)]


def _paths(paths):
    wide = np.zeros((B, T), np.int32)
    for b, p in enumerate(paths):
        wide[b, :len(p)] = p
    return _i32(wide), _i32([len(p) for p in paths])


@pytest.mark.parametrize("prefix", [0, 37])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_layer_step_against_the_definition(fmt, tree, prefix):
    say(f"[attention layer] format {fmt}, tree {tree}, prefix {prefix}")
    start = [70, 0, 21]
    L = Layer(fmt, start, prefix, seed=5)
    parent = _draft(3)[0] if tree else None
    L.step(L.start, parent)
    torch.cuda.synchronize()
    d, M = L.d, B * T
    # the projections: k and v stay in the fused rows, q has been rotated in place
    want = block.linear(L.inp["x"].reshape(M, HIDDEN), L.inp["w_in"]).reshape(M, N_Q + 2 * N_KV, D)
    assert _beyond_rounding(_f64(d["qkv"])[:, N_Q:], want[:, N_Q:]) < 1e-5
    q0 = torch.empty_like(d["qkv"])
    N = q0.shape[1] * D
    L.gdn.gdn_linear(d["x"], d["w_in"], M, N, HIDDEN, [(0, N, q0, N, 0)])
    q0 = _f64(q0)[:, :N_Q]
    f, m = ref.frequencies(ROT, THETA)
    pos = L.positions(L.start, parent).cpu().numpy()
    want = ref.rotate(q0, pos, ROT, f, m)
    q = _f64(d["q"])
    slack = 6.1e-7 * (np.abs(q0) + np.abs(np.roll(q0, ROT // 2, -1)) + np.abs(np.roll(q0, -ROT // 2, -1)))
    assert (np.abs(q - want) <= slack + 2.0 ** -8 * (np.abs(want) + slack)).all()
    # attention, on the cache's own values
    pk, pv = L.read(L.pages, 0, prefix) if prefix else (np.zeros((0, N_KV, D)),) * 2
    out = _f64(d["out"]).reshape(B, T, N_Q, D)
    for b in range(B):
        n = start[b] + T
        k, v = L.read(L.table[b], 0, n)
        sees = np.concatenate([np.ones((T, prefix + start[b]), bool), ref.sees(T, None if parent is None else parent[b])], 1)
        for h in range(N_KV):
            kk, vv = np.concatenate([pk[:, h], k[:, h]]), np.concatenate([pv[:, h], v[:, h]])
            for g in range(N_Q // N_KV):
                x = q.reshape(B, T, N_Q, D)[b, :, h * (N_Q // N_KV) + g]
                o, w = ref.attend(x, kk, vv, sees, D ** -0.5)
                e = (D + 8) * 2.0 ** -24 * D ** -0.5 * (np.abs(x) @ np.abs(kk).T).max()
                t = (w @ np.abs(vv)) * (2.0 ** -8 + 2 * e + len(kk) * 2.0 ** -24 + 2.0 ** -20)
                t = t + 2.0 ** -8 * (np.abs(o) + t)
                assert (np.abs(out[b, :, h * (N_Q // N_KV) + g] - o) <= t).all(), (b, h, g)
    want = block.linear(_f64(d["out"]).reshape(M, -1), L.inp["w_out"])
    assert _beyond_rounding(_f64(d["y"]).reshape(M, HIDDEN), want) < 1e-5


@pytest.mark.parametrize("fmt", [0, 1, 2])
def test_commit_leaves_what_a_straight_run_would(fmt):
    """Two rounds: a tree, its accepted path committed, a chain behind it; and beside it a cache that got the
    accepted tokens one after another.  A node's position is its depth, so both hold the same bits, and the
    second round gives the same."""
    from gated_deltanet_linear_verify_amd import gdn
    start = np.array([70, 0, 21], np.int32)
    L = Layer(fmt, start, seed=9)
    parent, paths = _draft(11)
    L.step(start, parent)
    rows = L.d["qkv"][:, N_Q:].clone()
    path, n_path = _paths(paths)
    gdn.gdn_kv_commit(L.kv, L.table, _i32(start), path, n_path, B, T)
    S = Layer(fmt, start, seed=9)
    keep = torch.zeros_like(rows)
    for b, p in enumerate(paths):
        keep[b * T:b * T + len(p)] = rows[[b * T + i for i in p]]
    gdn.gdn_kv_write(S.kv, keep[:, :N_KV], keep[:, N_KV:], S.table, _i32(start), n_path, B, T, rope=S.rope,
                     positions=S.positions(start))
    say("accepted", [len(p) for p in paths])
    assert len({len(p) for p in paths}) > 1 and any(p != list(range(len(p))) for p in paths)
    for b, p in enumerate(paths):
        for a, s in zip(L.read(L.table[b], 0, start[b] + len(p)), S.read(S.table[b], 0, start[b] + len(p))):
            assert (a == s).all(), b
    after = start + np.array([len(p) for p in paths], np.int32)
    for x in (L, S):
        x.d["x"].normal_(generator=torch.Generator("cuda").manual_seed(4))
        x.step(after)
    assert torch.equal(L.d["out"], S.d["out"]) and torch.equal(L.d["y"], S.d["y"])


def test_both_kinds_of_layer_in_one_graph():
    """A round of a GDN layer and a full-attention layer on one draft tree, with both commits, recorded once and
    replayed with other lengths, drafts and paths: bit for bit the eager round."""
    from gated_deltanet_linear_verify_amd import device, gdn
    shape = W.shape_with(W.MULTI_SLOT_VERIFY, n_kh=2, n_vh=4, n_pool=B, n_batch=B, n_tok=T)
    gin = W.make_tree_inputs(shape, 6)
    lay = device.upload(shape, gin, mode=gdn.GDN_TREE)
    L = Layer(gdn.GDN_KV_E4M3, [70, 0, 21], prefix=37, seed=2)
    d, M = L.d, B * T
    start, pos = _i32(np.zeros(B)), _i32(np.zeros((1, M)))
    parent, path, n_path, node = _i32(np.zeros((B, T))), _i32(np.zeros((B, T))), _i32(np.zeros(B)), _i32(np.zeros(B))
    lay["parent"] = parent
    pool = [t for t in (L.kv.k.view(torch.uint8), L.kv.v.view(torch.uint8), L.kv.k_scale, L.kv.v_scale, lay["state"], lay["conv_state"])]
    first = [t.clone() for t in pool]

    def round_():
        device.verify_tree(lay)
        device.attention_step(d, L.table, start, pos, None, parent, L.pages, L.plen)
        gdn.gdn_rollback_batch(lay["capture"], lay["slot_ids"], node, B)
        gdn.gdn_kv_commit(L.kv, L.table, start, path, n_path, B, T)

    def put(seed, at):
        p, paths = _draft(seed)
        a, n = _paths(paths)
        for t, x in ((start, _i32(at)), (pos, L.positions(np.array(at), p)), (parent, _i32(p)), (path, a), (n_path, n),
                     (node, _i32([q[-1] for q in paths]))):
            t.copy_(x)
        for t, x in zip(pool, first):
            t.copy_(x)
        for t in (d["y"], d["out"], lay["out"]):
            t.fill_(3.0)

    def result():
        torch.cuda.synchronize()
        return [t.clone() for t in (d["y"], d["out"], lay["out"], *pool)]

    put(1, [70, 0, 21])
    round_()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        round_()
    for seed, at in ((1, [70, 0, 21]), (2, [12, 48, 0]), (3, [0, 0, 0]), (4, [70, 15, 16])):
        put(seed, at)
        round_()
        want = result()
        put(seed, at)
        g.replay()
        for i, (a, w) in enumerate(zip(result(), want)):
            assert torch.equal(a, w), (seed, i)
