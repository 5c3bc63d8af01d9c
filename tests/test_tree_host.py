"""The operators of a verify round over trees without a GPU: the oracle against closed
forms and torch, and what the calls refuse before any GPU work."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P
from oracle import tree_oracle as T


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


END = [9, 4, 3, 4, 8, 7, 7, 8, 9]                    # 0 -> 1 -> {2, 3}, 0 -> 4 -> {5 -> 6, 7}, 0 -> 8


def test_oracle_trees_by_hand():
    assert T.parents(END) == [-1, 0, 1, 1, 0, 4, 5, 4, 0]
    a = T.ancestors(END)
    assert [np.flatnonzero(x).tolist() for x in a] == [[0], [0, 1], [0, 1, 2], [0, 1, 3], [0, 4], [0, 4, 5], [0, 4, 5, 6], [0, 4, 7], [0, 8]]
    n = len(END)
    for i in range(n):
        for j in range(n):
            assert a[i, j] == (j <= i < END[j])        # the interval form that the kernels use
    assert T.ancestors([3, 3, 3]).tolist() == np.tri(3, dtype=bool).tolist()


def test_oracle_walk_by_hand():
    draft = [0, 11, 12, 13, 14, 15, 16, 15, 11]
    assert T.accept(END, draft, [14, 0, 0, 0, 15, 16, 99, 0, 0], 9) == ([0, 4, 5, 6], [14, 15, 16, 99])
    assert T.accept(END, draft, [11, 13, 0, 7, 0, 0, 0, 0, 0], 9) == ([0, 1, 3], [11, 13, 7])      # the first child drafted so
    assert T.accept(END, draft, [14, 0, 0, 0, 15, 16, 99, 0, 0], 2) == ([0, 4], [14, 15])
    assert T.accept(END, draft, [5] * 9, 9) == ([0], [5]) and T.accept([], [], [], 4) == ([], [])


def test_oracle_walk_ends_before_a_row_with_nothing_to_draw():
    draft = [0, 11, 12, 13, 14, 15, 16, 15, -1]
    assert T.accept(END, draft, [14, 0, 0, 0, 15, -1, 99, 0, 0], 9) == ([0, 4], [14, 15])
    assert T.accept(END, draft, [-1] * 9, 9) == ([], []) and T.accept(END, draft, [-1, 0, 0, 0, 0, 0, 0, 0, 7], 9) == ([], [])


def test_oracle_attention_of_a_path_is_the_chain_s():
    """A node's row is what causal attention gives it when only its path has been appended."""
    r = np.random.default_rng(2)
    ps, n, old, hd = 8, len(END), 13, 8
    pages = 3
    c = {"k": r.standard_normal((pages, 2, ps, hd)), "v": r.standard_normal((pages, 2, ps, hd)), "pos": np.zeros((pages, 2, ps), np.int32),
         "weight": np.zeros((pages, 2, ps)), "table": np.array([[2, 0, 1]]), "length": np.array([old + n])}
    depth = T.ancestors(END).sum(1) - 1
    where = P.rows_of(c, 0)
    for i, (p, j) in enumerate(where):
        c["pos"][p, :, j] = i if i < old else old + depth[i - old]
    q = r.standard_normal((n, 4, hd))
    q_pos = old + depth
    out, lse, _ = T.attention(c, q, q_pos, [0, n], END, 0.3)
    for i in range(n):
        path = np.flatnonzero(T.ancestors(END)[i])
        rows = where[:old] + [where[old + j] for j in path]
        k = np.stack([c["k"][p, :, j] for p, j in rows], 1).repeat(2, 0)
        v = np.stack([c["v"][p, :, j] for p, j in rows], 1).repeat(2, 0)
        t = np.einsum("hd,hld->hl", q[i], k) * 0.3
        w = np.exp(t - t.max(1, keepdims=True))
        np.testing.assert_allclose(out[i], np.einsum("hl,hld->hd", w / w.sum(1, keepdims=True), v), rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(lse[i], torch.logsumexp(torch.tensor(t), 1).numpy(), rtol=1e-12)


def test_oracle_sampling_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [T.sample(l, u)[0] for u in (0.0, 0.05, 0.15, 0.49, 0.51, 0.69, 0.71, 0.99, 1.0, math.nan)] == [0, 0, 1, 1, 2, 2, 3, 3, 3, 0]
    assert T.sample(l, 0.4, top_k=2)[:2] == (1, pytest.approx(4 / 7)) and T.sample(l, 0.6, top_k=2)[:2] == (3, pytest.approx(3 / 7))
    assert T.sample(l, 0.99, top_p=0.69)[0] == 3 and T.sample(l, 0.99, top_p=0.39)[0] == 1 and T.sample(l, 0.5, top_p=0.0)[:2] == (1, 1.0)
    assert T.sample(l, 0.99, top_k=3, top_p=0.8)[0] == 3 and T.sample(l, 0.99, top_k=3, top_p=0.75)[:2] == (3, pytest.approx(3 / 7))
    assert T.sample(l, 0.99, min_p=0.6)[0] == 3 and T.sample(l, 0.99, min_p=0.8)[0] == 1 and T.sample(l, 0.3, min_p=5)[0] == 1
    assert T.sample(l, 0.3, temperature=0)[:2] == (1, 1.0) and T.sample(l, 0.7, temperature=math.inf)[:2] == (2, 0.25)
    p = T.sample(l, 0.2, temperature=0.5)[1]
    assert p == pytest.approx(0.16 / 0.30)
    eq = np.zeros(5)
    assert [T.sample(eq, 0.99, top_k=k)[0] for k in (1, 2, 5, 9)] == [0, 1, 4, 4] and T.sample(eq, 0.99, top_p=0.5)[0] == 2
    bad = np.array([math.nan, -math.inf, 1.0, math.inf])
    assert T.sample(bad, 0.9)[0] == 3 and T.sample(np.array([math.nan, -math.inf]), 0.5)[:2] == (-1, 0.0)


@pytest.mark.parametrize("seed", range(4))
def test_oracle_sampling_draws_torch_s_distribution(seed):
    """Uniforms on a grid fall on each token as often as its probability says."""
    r = np.random.default_rng(seed)
    l = r.standard_normal(30) * 2
    want = torch.softmax(torch.tensor(l) / 0.7, 0)
    top = want.sort(descending=True)
    keep = top.indices[: int(((top.values.cumsum(0) - top.values) < 0.8).sum())]
    p = torch.zeros(30, dtype=torch.float64)
    p[keep] = want[keep] / want[keep].sum()
    got = np.bincount([T.sample(l, (i + 0.5) / 4000, 0.7, 0, 0.8)[0] for i in range(4000)], minlength=30) / 4000
    assert np.abs(got - p.numpy()).max() <= 1 / 4000


@pytest.mark.parametrize("counts", [[3, 0], [1, 4]])
def test_oracle_commit_leaves_what_is_elsewhere(counts):
    r = np.random.default_rng(5)
    c = {"k": r.standard_normal((4, 1, 8, 8)), "v": r.standard_normal((4, 1, 8, 8)), "pos": r.integers(0, 99, (4, 1, 8)), "weight": r.random((4, 1, 8)),
         "table": np.array([[1, 3], [2, 0]]), "length": np.array([6 + counts[0], 3 + counts[1]])}
    before = {n: c[n].copy() for n in ("k", "v", "pos", "weight")}
    path = [[0, 2, 5, -1], [0, 1, 3, 6]]
    T.commit(c, path, counts)
    flat = lambda x, s: x[c["table"][s]][:, 0].reshape(16, -1)  # noqa: E731
    for n in before:
        for s, base in ((0, 6), (1, 3)):
            want = flat(before[n], s).copy()
            want[base:base + counts[s]] = flat(before[n], s)[[base + p for p in path[s][: counts[s]]]]
            assert (flat(c[n], s) == want).all()


# ---- refusals ------------------------------------------------------------------------


def refused(B, call, match=None, **args):
    """Refused for its arguments, with the host's tensors: the binding's own refusal of those is left out, so that the C
    side's checks are reached (nothing is launched)."""
    with pytest.MonkeyPatch.context() as m:
        if not torch.cuda.is_available():
            m.setattr(B.PagedCache, "_launch", lambda self, c, stream, *a: self._check(c(self._c, *a, None)))

            def direct(c, device, stream, a):
                rc = c(a, None)
                if rc:
                    raise B.DFlashError(rc, B.last_error(None))
            m.setattr(B, "_call_on", direct)
        with pytest.raises(B.DFlashError, match=match) as e:
            call(**args)
    assert e.value.code in (B.EINVAL, B.ERANGE)


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def sample_args(**over):
    return {**dict(logits=torch.zeros(3, 50), uniform=torch.zeros(3), token=ints(3)), **over}


@pytest.mark.parametrize("over", [
    dict(logits=torch.zeros(150)), dict(logits=torch.zeros(3, 50, dtype=torch.float16)), dict(logits=torch.zeros(3, 50, dtype=torch.float64)),
    dict(logits=torch.zeros(50, 3).T), dict(logits=torch.zeros(3, 100)[:, ::2]), dict(logits=torch.zeros(1, 50).expand(3, 50)), dict(logits=torch.zeros(3, 0)),
    dict(logits=torch.zeros(1, 1).expand(3, (1 << 20) + 1)), dict(uniform=torch.zeros(2)), dict(uniform=torch.zeros(3, dtype=torch.float64)),
    dict(uniform=torch.zeros(6)[::2]), dict(token=torch.zeros(3, dtype=torch.int64)), dict(token=ints(3, 1)), dict(prob=torch.zeros(3, dtype=torch.bfloat16)),
    dict(temperature=torch.zeros(1)), dict(top_k=torch.zeros(3)), dict(top_p=torch.zeros(4)), dict(min_p=ints(3)),
])
def test_sample_refuses(B, over):
    refused(B, B.sample, **sample_args(**over))


def test_sample_of_host_tensors_is_refused(B):
    with pytest.raises(B.DFlashError, match="not on a GPU"):
        B.sample(**sample_args())
    with pytest.raises(B.DFlashError, match="not on a GPU"):
        B.tree_accept(**accept_args())


def accept_args(**over):
    return {**dict(tree_end=ints(6), start=ints(3), draft=ints(6), sampled=ints(6), tokens=ints(2, 4), path=ints(2, 4), count=ints(2), length=ints(2)), **over}


@pytest.mark.parametrize("over", [
    dict(tree_end=ints(5)), dict(tree_end=torch.zeros(6)), dict(start=ints(1)), dict(draft=ints(7)), dict(sampled=torch.zeros(6, dtype=torch.int64)),
    dict(tokens=ints(2, 5)), dict(tokens=ints(4, 2).T), dict(path=ints(8)), dict(path=ints(2, 0), tokens=ints(2, 0)), dict(count=ints(3)), dict(length=ints(3)),
    dict(length=None, length_out=ints(2)), dict(length_out=ints(1)), dict(start=torch.zeros(65538, dtype=torch.int32)),
])
def test_accept_refuses(B, over):
    refused(B, B.tree_accept, **accept_args(**over))


def attention_args(**over):
    a = dict(q=torch.zeros(5, 4, 64, dtype=torch.bfloat16), q_pos=ints(5), start=ints(4), tree_end=ints(5), out=torch.zeros(5, 4, 64, dtype=torch.bfloat16),
             workspace=torch.zeros(1 << 24, dtype=torch.uint8))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(tree_end=ints(4)), dict(tree_end=torch.zeros(5)), dict(tree_end=ints(10)[::2]), dict(q=torch.zeros(5, 4, 64)), dict(q=torch.zeros(5, 5, 64, dtype=torch.bfloat16)),
    dict(q_pos=ints(4)), dict(out=torch.zeros(5, 4, 64)), dict(scale=0.0), dict(softcap=-1.0), dict(max_len=-1), dict(lse=torch.zeros(5, 3)), dict(window=1 << 40),
    dict(workspace=torch.zeros(1 << 20)),
])
def test_tree_attention_refuses(B, over):
    refused(B, B.PagedCache.allocate(80, 64, 2, 64, 3, 20, device="cpu").tree_attention, **attention_args(**over))


def test_tree_attention_refuses_a_small_workspace(B):
    c = B.PagedCache.allocate(80, 64, 2, 64, 3, 20, dtype="f32", device="cpu")
    refused(B, c.tree_attention, "workspace", **attention_args(q=torch.zeros(5, 4, 64), out=torch.zeros(5, 4, 64), workspace=torch.zeros(4, dtype=torch.uint8)))


@pytest.mark.parametrize("what", ["none", "sizes", "type", "width", "path", "count", "many", "twice"])
def test_commit_refuses(B, what):
    make = lambda **o: B.PagedCache.allocate(**{**dict(n_pages=4, page_rows=16, kv_heads=2, head_dim=64, n_seq=3, max_pages=2), **o}, device="cpu")  # noqa: E731
    a = dict(caches=[make(), make()], path=ints(3, 4), count=ints(3))
    if what == "none":
        a["caches"] = []
    elif what == "sizes":
        a["caches"][1] = make(kv_heads=4)
    elif what == "type":
        a["caches"][1] = make(dtype="f32")
    elif what == "width":
        a["path"] = ints(3, 0)
    elif what == "path":
        a["path"] = ints(2, 4)
    elif what == "count":
        a["count"] = torch.zeros(3, dtype=torch.int64)
    elif what == "many":
        a["caches"] = a["caches"][:1] * 1025
    else:
        a["caches"][1] = a["caches"][0]                  # a row that moves twice would be lost
    refused(B, B.paged_tree_commit, **a)


@pytest.mark.parametrize("what", ["k", "v", "pos", "weight", "k as v", "k as its own v", "part", "pos as weight"])
def test_commit_refuses_arrays_that_overlap(B, what):
    """All caches are moved at once: a row that is in two arrays would move twice."""
    shape, pages = (4, 2, 16), 4
    t = [{"k": torch.zeros(*shape, 64), "v": torch.zeros(*shape, 64), "pos": ints(*shape), "weight": torch.zeros(shape)} for _ in range(60)]
    if what in t[0]:
        t[57][what] = t[3][what]                         # (of another launch, too)
    elif what == "k as v":
        t[1]["v"] = t[0]["k"]
    elif what == "k as its own v":
        t[2]["v"] = t[2]["k"]
    elif what == "part":
        pool = torch.zeros(2 * pages - 1, *shape[1:], 64)
        t[0]["k"], t[1]["k"] = pool[:pages], pool[pages - 1:]
    else:
        t[5]["pos"] = t[7]["weight"].view(torch.int32)
    caches = [B.PagedCache(x["k"], x["v"], x["pos"], ints(3, 2), ints(3), weight=x["weight"]) for x in t]
    refused(B, B.paged_tree_commit, "overlap", caches=caches, path=ints(3, 4), count=ints(3))


def test_structs_are_the_header_s(B, tmp_path):
    """The packed layouts against the C compiler's."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    fields = {"dflash_sample_args": "logits uniform temperature top_k top_p min_p token prob logit_stride rows vocab dtype reserved",
              "dflash_tree_accept_args": "tree_end start draft sampled tokens path count length length_out rows n_seq width reserved",
              "dflash_paged_tree_commit_args": "path count weight_host width n_caches"}
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"dflash.h\"\nint main(void) {\n"
    for t, names in fields.items():
        src += "".join(f'printf("%zu ", offsetof({t}, {n}));' for n in names.split()) + f'printf("%zu\\n", sizeof({t}));\n'
    (tmp_path / "o.c").write_text(src + "return 0; }\n")
    from conftest import ROOT
    subprocess.run([cc, "-I", f"{ROOT}/include", str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = [[int(x) for x in line.split()] for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines()]

    def layout(f):
        at, out = 0, []
        for n, kind in __import__("re").findall(r"(\d*)([Qqi])", f.format):
            for _ in range(int(n or 1)):
                out.append(at)
                at += {"Q": 8, "q": 8, "i": 4}[kind]
        return out + [at]

    assert got == [layout(B._SAMPLE), layout(B._TREE_ACCEPT), layout(B._TREE_COMMIT)]


def test_c_calls_refuse_null_and_misaligned(B):
    x = torch.zeros(64)
    p = x.data_ptr()
    assert B.lib.dflash_sample(None, None) == B.EINVAL and B.lib.dflash_tree_accept(None, None) == B.EINVAL
    assert B.lib.dflash_paged_tree_commit(None, None, None) == B.EINVAL and B.lib.dflash_paged_tree_attention(None, None, None, None) == B.EINVAL
    names = ("logits", "uniform", "temperature", "top_k", "top_p", "min_p", "token", "prob")
    for i, n in enumerate(names):
        at = [p] * 8
        at[i] = p + 2
        assert B.lib.dflash_sample(B._SAMPLE.pack(*at, 4, 1, 4, B.F32, 0), None) == B.EINVAL and f"{n} is not 4-byte" in B.last_error()
        if n in ("logits", "uniform", "token"):
            at[i] = 0
            assert B.lib.dflash_sample(B._SAMPLE.pack(*at, 4, 1, 4, B.F32, 0), None) == B.EINVAL and f"{n} is NULL" in B.last_error()
    for bad in ((4, -1, 4, B.F32, 0), (4, 1, 0, B.F32, 0), (4, 1, 4, 7, 0), (3, 1, 4, B.F32, 0), (1 << 40, 1, 4, B.F32, 0), (4, (1 << 27) + 1, 4, B.F32, 0)):
        assert B.lib.dflash_sample(B._SAMPLE.pack(*[p] * 8, *bad), None) in (B.EINVAL, B.ERANGE)
    for i, n in enumerate(("tree_end", "start", "draft", "sampled", "tokens", "path", "count", "length", "length_out")):
        at = [p] * 9
        at[i] = p + 1
        assert B.lib.dflash_tree_accept(B._TREE_ACCEPT.pack(*at, 4, 1, 4, 0), None) == B.EINVAL and f"{n} is not 4-byte" in B.last_error()
        at[i] = 0
        assert B.lib.dflash_tree_accept(B._TREE_ACCEPT.pack(*at, 4, 1, 4, 0), None) == B.EINVAL
    for bad in ((-1, 1, 4, 0), (4, 0, 4, 0), (4, 65536, 4, 0), (4, 1, 0, 0), (4, 1, (1 << 20) + 1, 0), (4, 65535, 1 << 16, 0)):
        assert B.lib.dflash_tree_accept(B._TREE_ACCEPT.pack(*[p] * 9, *bad), None) in (B.EINVAL, B.ERANGE)
    assert B.lib.dflash_sample(B._SAMPLE.pack(0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 4, B.F32, 0), None) == B.OK      # no rows
    assert B.last_error() != ""
