"""The paged-cache operators without a GPU: the oracle against closed forms and
torch fp64, and what the calls refuse before any GPU work."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as P


@pytest.fixture(scope="module")
def B():
    from block_speculative_decoding_dflash_gb300 import build
    build.build()
    from block_speculative_decoding_dflash_gb300 import binding
    return binding


def small(seed=0, n_seq=2, length=(7, 20), nkv=2, hd=8, ps=8, width=3):
    r = np.random.default_rng(seed)
    n_pages = n_seq * width + 1
    return {"k": r.standard_normal((n_pages, nkv, ps, hd)), "v": r.standard_normal((n_pages, nkv, ps, hd)),
            "pos": np.zeros((n_pages, nkv, ps), dtype=np.int32), "weight": r.random((n_pages, nkv, ps)),
            "table": r.permutation(n_pages)[: n_seq * width].reshape(n_seq, width).astype(np.int32),
            "length": np.array(length, dtype=np.int32)}


def test_oracle_attention_is_torch_attention():
    c = small()
    r = np.random.default_rng(1)
    for s in range(2):
        for i, (page, row) in enumerate(P.rows_of(c, s)):
            c["pos"][page, :, row] = i
    start = np.array([0, 3, 5])
    q = r.standard_normal((5, 4, 8))
    q_pos = np.array([4, 5, 6, 18, 19])
    out, lse, _ = P.attention(c, q, q_pos, start, 0.3)
    for s in range(2):
        rows = P.rows_of(c, s)
        k = torch.tensor(np.stack([c["k"][p, :, j] for p, j in rows], 1)).repeat_interleave(2, 0)
        v = torch.tensor(np.stack([c["v"][p, :, j] for p, j in rows], 1)).repeat_interleave(2, 0)
        new = slice(start[s], start[s + 1])
        mask = torch.arange(len(rows))[None] <= torch.tensor(q_pos[new])[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q[new]).transpose(0, 1), k, v, attn_mask=mask, scale=0.3)
        np.testing.assert_allclose(out[new], want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-13)
        t = torch.tensor(q[new]).transpose(0, 1) @ k.transpose(1, 2) * 0.3
        want = torch.logsumexp(t.masked_fill(~mask, -math.inf), -1)
        np.testing.assert_allclose(lse[new], want.T.numpy(), rtol=1e-12)


def test_oracle_masks_by_hand():
    pq, pk = np.array([[5], [9]]), np.array([[0, 4, 5, 6, 9]])
    assert P.sees(pq, pk, True, 0, None).tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 1]]
    assert P.sees(pq, pk, True, 3, None).tolist() == [[0, 1, 1, 0, 0], [0, 0, 0, 1, 1]]
    assert P.sees(pq, pk, False, 1, None).tolist() == [[0, 1, 1, 1, 0], [0, 0, 0, 0, 1]]
    assert P.sees(pq, pk, True, 1, 1).tolist() == [[1, 1, 1, 0, 0], [1, 0, 0, 0, 1]]


def test_oracle_weights_sum_to_the_queries_that_see_something():
    c = small(3)
    c["pos"][:] = np.arange(8)[None, None]
    start, q_pos = np.array([0, 2, 4]), np.array([7, 7, 7, -1])
    q = np.random.default_rng(2).standard_normal((4, 4, 8))
    _, lse, _ = P.attention(c, q, q_pos, start, 0.4, softcap=3.0, slopes=np.array([0.1, 0.2, 0.3, 0.4]))
    assert np.isneginf(lse[3]).all()
    w, _ = P.key_weight(c, q, q_pos, start, lse, None, 1.0, np.zeros(c["pos"].shape), 0.4, softcap=3.0, slopes=np.array([0.1, 0.2, 0.3, 0.4]))
    np.testing.assert_allclose(w.sum(), 3 * 4, rtol=1e-12)


def test_oracle_rotation_is_a_complex_turn_and_keeps_relative_positions():
    r = np.random.default_rng(4)
    x, y = r.standard_normal((1, 12)), r.standard_normal((1, 12))
    for neox in (True, False):
        z = P.rotate(x, [3], bytes(4), 100.0, neox)
        a = x[0, :8].reshape(2, 4) if neox else x[0, :8].reshape(4, 2).T
        want = (a[0] + 1j * a[1]) * np.exp(1j * 3 * 100.0 ** (-np.arange(4) / 4))
        got = z[0, :8].reshape(2, 4) if neox else z[0, :8].reshape(4, 2).T
        np.testing.assert_allclose(got[0] + 1j * got[1], want, rtol=1e-12)
        assert (z[0, 8:] == x[0, 8:]).all()
        axes = bytes([0, 1, 2, 0, 1, 2])
        one = P.rotate(x, [9, 5, 1], axes, 50.0, neox) @ P.rotate(y, [7, 1, 4], axes, 50.0, neox).T
        two = P.rotate(x, [29, 15, 11], axes, 50.0, neox) @ P.rotate(y, [27, 11, 14], axes, 50.0, neox).T
        np.testing.assert_allclose(one, two, rtol=1e-10)


def test_oracle_eviction_by_hand():
    c = small(5, n_seq=1, length=(6,), nkv=1, ps=8, width=1)
    page = int(c["table"][0, 0])
    c["weight"][page, 0] = [0.5, 0.1, 0.5, 0.9, np.nan, 0.5, 7, 7]
    c["pos"][page, 0] = [0, 1, 2, 3, 4, 5, 0, 0]
    k = c["k"].copy()
    w, p = np.zeros(c["weight"].shape), np.zeros(c["pos"].shape)
    # heaviest three: row 3, then rows 0 and 2 of the three at 0.5; row 3 moves into hole 1
    assert P.evict(c, 3, 0, [6], w, p).tolist() == [3]
    assert w[page, 0, :3].tolist() == [0.5, 0.9, 0.5] and p[page, 0, :3].tolist() == [0, 3, 2]
    assert (c["k"][page, 0, 1] == k[page, 0, 3]).all() and (c["k"][page, 0, 2:] == k[page, 0, 2:]).all()
    c["k"][:] = k
    # the last two positions first, the NaN among them; row 3 takes the last place
    assert P.evict(c, 3, 2, [6], w, p).tolist() == [3]
    assert p[page, 0, :3].tolist() == [3, 4, 5]


# ---- refusals ------------------------------------------------------------------------

@pytest.fixture(scope="module")
def cache(B):
    return B.PagedCache.allocate(8, 16, 2, 64, 3, 2, device="cpu")


def refused(B, call, args):
    """The call is refused for its arguments. These tensors are the host's; so that the C side's checks are reached too, the
    binding's own refusal of them is left out where there is no GPU that a launch could run on."""
    with pytest.MonkeyPatch.context() as m:
        if not torch.cuda.is_available():
            m.setattr(B.PagedCache, "_launch", lambda self, call, stream, *args: self._check(call(self._c, *args, None)))
        with pytest.raises(B.DFlashError) as e:
            call(**args)
    assert e.value.code in (B.EINVAL, B.ERANGE) and str(e.value)


def test_host_tensors_are_refused(B, cache):
    with pytest.raises(B.DFlashError, match="not on a GPU"):
        cache.append(**append_args())


def append_args(**over):
    a = dict(q=torch.zeros(5, 4, 64, dtype=torch.bfloat16), k=torch.zeros(5, 2, 64, dtype=torch.bfloat16), v=torch.zeros(5, 2, 64, dtype=torch.bfloat16),
             row_pos=torch.zeros(5, dtype=torch.int32), start=torch.zeros(4, dtype=torch.int32), q_out=torch.zeros(5, 4, 64, dtype=torch.bfloat16),
             rope_pos=torch.zeros(2, 5, dtype=torch.int32), pair_axis=bytes([0, 1] * 16))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(5, 4, 64)), dict(q=torch.zeros(5, 3, 64, dtype=torch.bfloat16), q_out=torch.zeros(5, 3, 64, dtype=torch.bfloat16)),
    dict(q=torch.zeros(5, 4, 32, dtype=torch.bfloat16)), dict(k=torch.zeros(5, 4, 64, dtype=torch.bfloat16)), dict(k=torch.zeros(4, 2, 64, dtype=torch.bfloat16)),
    dict(v=torch.zeros(5, 2, 65, dtype=torch.bfloat16)[:, :, :64]), dict(v=torch.zeros(2, 5, 64, dtype=torch.bfloat16).transpose(0, 1)),
    dict(row_pos=torch.zeros(5, dtype=torch.int64)), dict(start=torch.zeros(3, dtype=torch.int32)), dict(q_out=torch.zeros(5, 2, 64, dtype=torch.bfloat16)),
    dict(rope_pos=None), dict(rope_pos=torch.zeros(2, 4, dtype=torch.int32)), dict(pair_axis=bytes([0, 2])), dict(pair_axis=bytes(33)),
    dict(theta=0.5), dict(theta=math.nan), dict(eps=0.0), dict(q_norm=torch.zeros(64)), dict(k_norm=torch.zeros(32, dtype=torch.bfloat16)),
    dict(rope_pos=torch.zeros(5, 5, dtype=torch.int32), pair_axis=bytes(4)),
    dict(q=torch.zeros(5 * 256 + 8, dtype=torch.bfloat16)[1:5 * 256 + 1].view(5, 4, 64)),
    dict(q=torch.zeros(5, 260, dtype=torch.bfloat16)[:, :256].unflatten(1, (4, 64))),
])
def test_append_refuses(B, cache, over):
    refused(B, cache.append, append_args(**over))


def attention_args(**over):
    a = dict(q=torch.zeros(5, 4, 64, dtype=torch.bfloat16), q_pos=torch.zeros(5, dtype=torch.int32), start=torch.zeros(4, dtype=torch.int32),
             out=torch.zeros(5, 4, 64, dtype=torch.bfloat16), workspace=torch.zeros(1 << 24, dtype=torch.uint8))
    return {**a, **over}


@pytest.mark.parametrize("over", [
    dict(q=torch.zeros(5, 4, 64)), dict(q=torch.zeros(5, 5, 64, dtype=torch.bfloat16)), dict(out=torch.zeros(5, 4, 64)), dict(q_pos=torch.zeros(4, dtype=torch.int32)),
    dict(start=torch.zeros(4, dtype=torch.int64)), dict(lse=torch.zeros(5, 3)), dict(lse=torch.zeros(4, 5).T), dict(slopes=torch.zeros(2)), dict(prefix=torch.zeros(2, dtype=torch.int32)),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(softcap=-1.0), dict(softcap=math.nan), dict(softcap=math.inf), dict(max_len=-1),
    dict(workspace=torch.zeros(1 << 20)), dict(window=1 << 40), dict(scale="wide"), dict(softcap=1e300),
    dict(scale=1e19), dict(softcap=1e-19), dict(softcap=1e19),
])
def test_attention_refuses(B, over):
    c = B.PagedCache.allocate(80, 64, 2, 64, 3, 20, device="cpu")
    refused(B, c.attention, attention_args(**over))


def test_attention_refuses_a_small_workspace(B):
    c = B.PagedCache.allocate(80, 64, 2, 64, 3, 20, dtype="f32", device="cpu")
    args = attention_args(q=torch.zeros(5, 4, 64), out=torch.zeros(5, 4, 64), workspace=torch.zeros(4, dtype=torch.uint8))
    refused(B, c.attention, args)


@pytest.mark.parametrize("over", [dict(lse=None), dict(lse=torch.zeros(5, 2)), dict(weight=torch.zeros(8, 2, 8)), dict(weight_out=torch.zeros(8, 2, 16, dtype=torch.float64)),
                                  dict(decay=math.nan), dict(scale=0.0)])
def test_key_weight_refuses(B, cache, over):
    a = attention_args(lse=torch.zeros(5, 4))
    del a["out"], a["workspace"]
    refused(B, cache.key_weight, {**a, **over})


@pytest.mark.parametrize("over", [dict(budget=0), dict(recent=-1), dict(budget=1 << 32), dict(recent=0.5), dict(next_pos=torch.zeros(2, dtype=torch.int32)), dict(weight_out=torch.zeros(1)),
                                  dict(length_out=torch.zeros(3, dtype=torch.int64)), dict(workspace=torch.zeros(3, dtype=torch.uint8))])
def test_evict_refuses(B, cache, over):
    refused(B, cache.evict, {**dict(budget=4, recent=1, next_pos=torch.zeros(3, dtype=torch.int32)), **over})


@pytest.mark.parametrize("over", [dict(page_rows=12), dict(page_rows=4), dict(page_rows=8192), dict(head_dim=4), dict(head_dim=20), dict(head_dim=264),
                                  dict(max_pages=(1 << 16) + 1), dict(n_seq=0), dict(n_pages=0)])
def test_cache_refuses(B, over):
    with pytest.raises(B.DFlashError):
        B.PagedCache.allocate(**{**dict(n_pages=1, page_rows=16, kv_heads=1, head_dim=64, n_seq=1, max_pages=1), **over}, device="cpu")


def test_structs_are_the_header_s(B, tmp_path):
    """The packed layouts against the C compiler's."""
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    fields = {"dflash_paged_cache": "k v pos table length status n_pages page_rows kv_heads head_dim n_seq max_pages dtype",
              "dflash_paged_append_args": "q k v row_pos start rope_pos pair_axis_host q_norm k_norm q_out weight q_stride k_stride v_stride rows "
                                          "n_q_heads n_axes rot_pairs rope_neox rope_theta rms_eps",
              "dflash_paged_attention_args": "q q_pos start slopes prefix out lse q_stride rows n_q_heads causal window max_len scale softcap reserved "
                                             "workspace workspace_bytes",
              "dflash_paged_evict_args": "weight next_pos weight_out pos_out length_out budget recent workspace workspace_bytes"}
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"dflash.h\"\nint main(void) {\n"
    for t, names in fields.items():
        src += "".join(f'printf("%zu ", offsetof({t}, {n}));' for n in names.split()) + f'printf("%zu\\n", sizeof({t}));\n'
    (tmp_path / "o.c").write_text(src + "return 0; }\n")
    from conftest import ROOT
    subprocess.run([cc, "-I", f"{ROOT}/include", str(tmp_path / "o.c"), "-o", str(tmp_path / "o")], check=True)
    got = [[int(x) for x in line.split()] for line in subprocess.run([str(tmp_path / "o")], capture_output=True, text=True, check=True).stdout.splitlines()]

    def layout(*formats):
        at, out = 0, []
        for f in formats:
            for n, kind in __import__("re").findall(r"(\d*)([a-zA-Z])", f.format.lstrip("=")):
                for _ in range(int(n or 1)):
                    if kind != "x":
                        out.append(at)
                    at += {"Q": 8, "q": 8, "i": 4, "f": 4, "x": 1}[kind]
        return out + [at]

    assert got == [layout(B._PAGED_CACHE), layout(B._PAGED_APPEND), layout(B._PAGED_ATTENTION, B._PAGED_WORKSPACE), layout(B._PAGED_EVICT, B._PAGED_WORKSPACE)]


def test_c_calls_refuse_null(B):
    n = ctypes.c_int64()
    assert B.lib.dflash_paged_append(None, None, None) == B.EINVAL
    assert B.lib.dflash_paged_attention(None, None, None) == B.EINVAL
    assert B.lib.dflash_paged_key_weight(None, None, None, 1.0, None, None) == B.EINVAL
    assert B.lib.dflash_paged_evict(None, None, None) == B.EINVAL
    assert B.lib.dflash_paged_attention_workspace(None, None, ctypes.byref(n)) == B.EINVAL
    assert B.lib.dflash_paged_evict_workspace(None, None, None) == B.EINVAL
    assert B.last_error() != ""


def test_misaligned_arrays_are_refused(B):
    """Addresses within an element, and of arrays read 16 bytes at a time within those (nothing is launched: the checks come first)."""
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    rows = torch.zeros(4, 2, 16)
    at = {n: k.data_ptr() if n in ("k", "v", "q", "out") else rows.data_ptr() for n in
          ("k", "v", "pos", "table", "length", "status", "q", "q_pos", "start", "slopes", "prefix", "out", "lse", "workspace", "next_pos", "weight", "pos_out", "length_out")}

    def cache(**a):
        a = {**at, **a}
        return B._PAGED_CACHE.pack(*(a[n] for n in ("k", "v", "pos", "table", "length", "status")), 4, 16, 2, 64, 1, 1, B.BF16)

    def attention(**a):
        a = {**at, **a}
        args = B._PAGED_ATTENTION.pack(*(a[n] for n in ("q", "q_pos", "start", "slopes", "prefix", "out", "lse")), 256, 1, 4, 1, 0, 0, 0.1, 0.0, 0)
        return B.lib.dflash_paged_attention_workspace(cache(), args + B._NO_WORKSPACE, ctypes.byref(ctypes.c_int64()))

    def evict(**a):
        a = {**at, **a}
        args = B._PAGED_EVICT.pack(*(a[n] for n in ("weight", "next_pos", "weight", "pos_out", "length_out")), 4, 0)
        return B.lib.dflash_paged_evict(cache(), args + B._PAGED_WORKSPACE.pack(at["workspace"], 0), None)

    def workspace_of(**a):
        return B.lib.dflash_paged_attention_workspace(cache(**a), B._PAGED_ATTENTION.pack(*(at[n] for n in ("q", "q_pos", "start", "slopes", "prefix", "out", "lse")),
                                                                                         256, 1, 4, 1, 0, 0, 0.1, 0.0, 0) + B._NO_WORKSPACE, ctypes.byref(ctypes.c_int64()))

    assert attention() == 0 and workspace_of() == 0
    for call, names, wide in ((workspace_of, ("table", "length", "status"), ("k", "v", "pos")), (attention, ("q_pos", "start", "slopes", "prefix", "lse"), ("q", "out")),
                              (evict, ("next_pos", "length_out"), ("weight", "pos_out"))):
        for n in names:
            for off in (1, 2):
                assert call(**{n: at[n] + off}) == B.EINVAL and f"{n} is not 4-byte aligned" in B.last_error().replace("cache.", "")
            if call is not evict:                        # (whose workspace is too small here: nothing runs)
                assert call(**{n: at[n] + 4}) == 0
            else:
                assert call(**{n: at[n] + 4}) == B.EINVAL and "workspace" in B.last_error()
        for n in wide:
            assert call(**{n: at[n] + 8}) == B.EINVAL and "16-byte aligned" in B.last_error()
