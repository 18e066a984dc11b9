"""Arguments that the tree and cache-page entry points refuse on the host,
before any launch (no GPU needed but where marked)."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK, INVALID, WORKSPACE = 0, 1, 3
A = P(1 << 20)                  # an aligned address that nothing reads
ODD = P((1 << 20) + 8)
ODDER = P((1 << 20) + 2)


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def _change(base, **kw):
    a = dict(base)
    a.update(kw)
    return list(a.values())


def _pools(*sizes, at=1 << 20):
    return (ctypes.c_void_p * len(sizes))(*[at] * len(sizes)), (ctypes.c_int64 * len(sizes))(*sizes)


def _with_pools(base, at=1 << 20, sizes=(73728, 16)):
    a = dict(base)
    a["pools"], a["bytes"] = _pools(*sizes, at=at)
    a["n_pools"] = len(sizes)
    return a


TREE = dict(q=A, qd=0, qs=1.0, kv=A, kd=0, ks=1.0, scales=P(0), sb=0, bt=A, lens=A, tl=P(0), mask=A, stride=3, B=2,
            q_len=3, H=16, mb=3, nb=5, sm=0.1, split=0, out=A, od=0, lse=A, ws=A, n=1 << 40, s=P(0))


@pytest.mark.parametrize("bad", [
    dict(B=0), dict(q_len=0), dict(q_len=65, stride=65), dict(H=0), dict(H=4097), dict(mb=0), dict(mb=(1 << 24) + 1),
    dict(nb=0), dict(nb=1 << 25), dict(sm=0.0), dict(sm=float("nan")), dict(split=-1), dict(q=P(0)), dict(kv=P(0)),
    dict(bt=P(0)), dict(lens=P(0)), dict(mask=P(0)), dict(out=P(0)), dict(lse=P(0)), dict(od=1), dict(q=ODD),
    dict(kv=ODD), dict(out=ODD), dict(ws=ODD), dict(mask=P((1 << 20) + 4)), dict(stride=2), dict(stride=-3),
    dict(qd=1), dict(kd=1), dict(qd=1, kd=1, qs=0.0), dict(qd=1, kd=1, ks=-1.0), dict(scales=A, sb=64),
    dict(qd=1, kd=1, scales=A, sb=0), dict(qd=1, kd=1, scales=A, sb=24)])
def test_tree(m, bad):
    assert m.lib.mla_decode_paged_tree(*_change(TREE, **bad)) == INVALID


COPY = dict(pools=None, bytes=None, n_pools=2, nb=5, src=A, dst=A, n=3, s=P(0))


def _bad_pools(base):
    for kw in (dict(sizes=(73728, 6)), dict(sizes=(0,)), dict(sizes=(-64,)), dict(sizes=((1 << 28) + 16,)),
               dict(at=(1 << 20) + 8, sizes=(1024,)), dict(at=(1 << 20) + 2, sizes=(16,)), dict(at=0, sizes=(16,)),
               dict(sizes=(16,) * 201)):
        yield _with_pools(base, **kw)
    yield {**_with_pools(base), "pools": None}
    yield {**_with_pools(base), "bytes": None}
    yield {**_with_pools(base), "n_pools": -1}


def test_copy(m):
    for bad in _bad_pools(COPY):
        assert m.lib.mla_cache_copy(*bad.values()) == INVALID
    for bad in (dict(nb=0), dict(nb=1 << 25), dict(n=-1), dict(n=(1 << 16) + 1), dict(n=1 << 25), dict(src=P(0)), dict(dst=P(0))):
        assert m.lib.mla_cache_copy(*_change(_with_pools(COPY), **bad)) == INVALID
    assert m.lib.mla_cache_copy(*_change(_with_pools(COPY), n=0, src=P(0), dst=P(0))) == OK
    assert m.lib.mla_cache_copy(*_change(COPY, n_pools=0)) == OK


RESIZE = dict(refs=A, nb=5, bt=A, lens=A, new=A, B=2, mb=3, s=P(0))
SEQS = [dict(refs=P(0)), dict(refs=ODD), dict(nb=0), dict(nb=1 << 25), dict(bt=P(0)), dict(lens=P(0)), dict(B=0),
        dict(B=8193), dict(mb=0), dict(mb=(1 << 24) + 1), dict(B=128, mb=1 << 24)]


@pytest.mark.parametrize("bad", SEQS + [dict(new=P(0))])
def test_resize(m, bad):
    assert m.lib.mla_cache_resize(*_change(RESIZE, **bad)) == INVALID


FORK = dict(pools=None, bytes=None, n_pools=2, rows=1, refs=A, nb=5, bt=A, lens=A, B=2, mb=3, parents=A, children=A, n=4,
            ws=A, size=48, s=P(0))


def test_fork(m):
    for bad in _bad_pools(FORK):
        assert m.lib.mla_cache_fork(*bad.values()) == INVALID
    for bad in SEQS + [dict(rows=-1), dict(rows=2), dict(rows=3), dict(n=-1), dict(n=8193), dict(parents=P(0)), dict(children=P(0)), dict(ws=ODDER)]:
        assert m.lib.mla_cache_fork(*_change(_with_pools(FORK), **bad)) == INVALID
    assert m.lib.mla_cache_fork(*_change(_with_pools(FORK), size=47)) == WORKSPACE
    assert m.lib.mla_cache_fork(*_change(_with_pools(FORK), ws=P(0))) == WORKSPACE
    assert m.lib.mla_cache_fork(*_change(_with_pools(FORK), n=0, parents=P(0), children=P(0), ws=P(0), size=0)) == OK
    n = ctypes.c_size_t(0)
    assert m.lib.mla_cache_fork_workspace_size(4, ctypes.byref(n)) == OK and n.value == 48
    assert m.lib.mla_cache_fork_workspace_size(-1, ctypes.byref(n)) == INVALID
    assert m.lib.mla_cache_fork_workspace_size(8193, ctypes.byref(n)) == INVALID
    assert m.lib.mla_cache_fork_workspace_size(1, None) == INVALID


COMPACT = dict(pools=None, bytes=None, n_pools=2, refs=A, nb=5, bt=A, lens=A, B=2, mb=3, live=A, ws=A, size=1 << 20,
               s=P(0))


def test_compact(m):
    for bad in _bad_pools(COMPACT):
        assert m.lib.mla_cache_compact(*bad.values()) == INVALID
    for bad in SEQS + [dict(live=P(0)), dict(ws=ODDER)]:
        assert m.lib.mla_cache_compact(*_change(_with_pools(COMPACT), **bad)) == INVALID
    n = ctypes.c_size_t(0)
    assert m.lib.mla_cache_compact_workspace_size(5, ctypes.byref(n)) == OK
    assert m.lib.mla_cache_compact(*_change(_with_pools(COMPACT), size=n.value - 1)) == WORKSPACE
    assert m.lib.mla_cache_compact(*_change(_with_pools(COMPACT), ws=P(0))) == WORKSPACE
    for bad in (0, 1 << 25):
        assert m.lib.mla_cache_compact_workspace_size(bad, ctypes.byref(n)) == INVALID
    assert m.lib.mla_cache_compact_workspace_size(1, None) == INVALID


ACCEPT = dict(pools=None, kd=0, scales=None, sb=0, n_pools=2, nb=5, bt=A, lens=A, tl=P(0), q_len=4, path=A, width=3,
              count=A, B=2, mb=3, new=P(1 << 21), s=P(0))


def test_accept(m):
    good = dict(ACCEPT)
    good["pools"], _ = _pools(1, 1)
    odd, _ = _pools(1, 1, at=(1 << 20) + 8)
    none, _ = _pools(1, 1, at=0)
    for bad in (dict(nb=0), dict(nb=1 << 25), dict(B=0), dict(mb=0), dict(mb=(1 << 24) + 1), dict(q_len=0),
                dict(q_len=65), dict(width=0), dict(width=65), dict(n_pools=-1), dict(n_pools=201), dict(kd=2),
                dict(bt=P(0)), dict(lens=P(0)), dict(path=P(0)), dict(count=P(0)), dict(new=P(0)), dict(new=A),
                dict(pools=None), dict(pools=odd), dict(pools=none), dict(scales=good["pools"], sb=64),
                dict(scales=good["pools"], sb=63, kd=1), dict(scales=none, sb=64, kd=1)):
        assert m.lib.mla_cache_accept(*_change(good, **bad)) == INVALID, bad


# ------------------------------------------------- the Python calls' checks
def _calls(m, dev):
    """One good set of arguments for each call, by name (sequences without tokens)."""
    def z(*s, dtype=torch.int32):
        return torch.zeros(s, dtype=torch.uint8 if dtype is E4M3 else dtype, device=dev).view(dtype)

    E4M3, BF = torch.float8_e4m3fn, torch.bfloat16
    seqs = dict(refs=z(3), block_table=z(2, 2), seq_lens=z(2))
    pools = [z(3, 64, 576, dtype=E4M3), torch.ones((3, 2), device=dev)]
    return {
        m.mla_decode_paged_tree: dict(q=z(2, 3, 4, 576, dtype=E4M3), kv_cache=pools[0], block_table=z(2, 2),
                                      seq_lens=z(2), tree_mask=z(2, 3, dtype=torch.int64), sm_scale=1.0,
                                      tree_lens=z(2), kv_scales=pools[1], out=z(2, 3, 4, 512, dtype=BF),
                                      lse=z(2, 3, 4, dtype=torch.float32)),
        m.mla_cache_copy: dict(pools=pools, src=z(2), dst=z(2)),
        m.mla_cache_resize: dict(**seqs, new_lens=z(2)),
        m.mla_cache_fork: dict(pools=pools, **seqs, parents=z(2), children=z(2) + 1),
        m.mla_cache_compact: dict(pools=pools, **seqs, n_live=z(1)),
        m.mla_cache_accept: dict(pools=[pools[0]] * 2, block_table=z(2, 2), seq_lens=z(2), path=z(2, 3),
                                 path_lens=z(2), q_len=3, tree_lens=z(2), kv_scales=[pools[1]] * 2, new_lens=z(2)),
    }


def test_tensors_of_the_host_and_other_things(m):
    for call, kw in _calls(m, "cpu").items():
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(**kw)
        with pytest.raises(TypeError, match="must be a tensor"):
            call(**{**kw, **{k: 3 for k in ("src", "refs", "block_table", "q") if k in kw}})
        with pytest.raises(TypeError):
            call()
    kw = _calls(m, "cpu")[m.mla_decode_paged_tree]
    with pytest.raises(TypeError, match="tree_mask"):
        m.mla_decode_paged_tree(**{**kw, "tree_mask": None})


@pytest.mark.gpu
def test_python_checks(m):
    """Every tensor in turn of another type, rank, device and stride, and of
    another length; numbers that are none."""
    for call, kw in _calls(m, "cuda").items():
        call(**kw)                              # as it stands it is taken
        for name, t in kw.items():
            if isinstance(t, list):
                for bad, errors in ((t[:1] + [t[0].cpu()], ValueError), (t[:1] + [3], TypeError), (5, TypeError),
                                    ([x[:1] for x in t[:1]] + t[1:], ValueError), (t * 101, ValueError),
                                    ([t[0].transpose(0, 1)], ValueError), ([t[0][:0]], ValueError)):
                    with pytest.raises(errors):
                        call(**{**kw, name: bad})
                continue
            if not isinstance(t, torch.Tensor):
                with pytest.raises(TypeError):
                    call(**{**kw, name: "x"})
                continue
            for bad, errors in ((t.unsqueeze(0).unsqueeze(0), ValueError), (t.cpu(), ValueError),
                                (torch.zeros(t.shape, dtype=torch.float64, device="cuda"), TypeError),
                                ([1], TypeError)):
                with pytest.raises(errors):
                    call(**{**kw, name: bad})
            if t.numel() > 1:
                wide = torch.zeros((*t.shape, 2), dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype,
                                   device="cuda").view(t.dtype)[..., 0]
                with pytest.raises(ValueError):
                    call(**{**kw, name: wide})
            if not (name == "refs" and call is m.mla_cache_resize):      # (any number of pages will do)
                with pytest.raises((ValueError, TypeError)):
                    call(**{**kw, name: t[:-1]})
    assert m.mla_get_device_error() in (0, 1, 16, 17)   # (the second child is the first one's: refused)


@pytest.mark.gpu
def test_other_python_refusals(m):
    calls = _calls(m, "cuda")
    kw = calls[m.mla_cache_accept]
    bf = torch.zeros((3, 64, 576), dtype=torch.bfloat16, device="cuda")
    for bad, error in ((dict(pools=[bf, bf]), TypeError), (dict(pools=[bf.float()], kv_scales=None), TypeError),
                       (dict(pools=[bf[:, :32].contiguous()], kv_scales=None), ValueError),
                       (dict(kv_scales=kw["kv_scales"][:1]), ValueError),
                       (dict(kv_scales=[torch.ones((3, 3), device="cuda")] * 2), ValueError),
                       (dict(kv_scales=[kw["kv_scales"][0], torch.ones((3, 4), device="cuda")]), ValueError)):
        with pytest.raises(error):
            m.mla_cache_accept(**{**kw, **bad})
    for bad in (dict(q_len=0), dict(q_len=65), dict(new_lens=kw["seq_lens"])):
        with pytest.raises(m.MlaError) as e:
            m.mla_cache_accept(**{**kw, **bad})
        assert e.value.status == INVALID and "mla_cache_accept" in str(e.value)
    kw = calls[m.mla_cache_fork]
    with pytest.raises(m.MlaError) as e:
        m.mla_cache_fork(**{**kw, "workspace": torch.zeros(8, dtype=torch.uint8, device="cuda")})
    assert e.value.status == WORKSPACE
    with pytest.raises(m.MlaError):                   # refs off its 16 bytes
        m.mla_cache_resize(**{**calls[m.mla_cache_resize], "refs": torch.zeros(4, dtype=torch.int32, device="cuda")[1:]})
    kw = calls[m.mla_decode_paged_tree]
    with pytest.raises(ValueError):
        m.mla_decode_paged_tree(**{**kw, "tree_mask": kw["tree_mask"][0, :2].contiguous()})
    with pytest.raises(ValueError):
        m.mla_cache_copy(calls[m.mla_cache_copy]["pools"] * 101, *[kw["seq_lens"]] * 2)
    assert m.mla_cache_copy([], kw["seq_lens"], kw["seq_lens"]) is None
    m.mla_get_device_error()


def test_tree_workspace(m):
    n = ctypes.c_size_t(0)
    size = m.lib.mla_decode_tree_workspace_size
    assert size(2, 8, 16, 64 * 99, 0, ctypes.byref(n)) == OK and n.value > 8
    assert m.mla_decode_tree_workspace_size(2, 8, 16, 64 * 99) == n.value
    assert size(2, 8, 16, 64 * 3, 0, ctypes.byref(n)) == OK and n.value == 0
    assert size(2, 8, 16, 64 * 3, 2, ctypes.byref(n)) == OK and n.value > 0
    for bad in ((0, 1, 16, 64, 0), (1, 65, 16, 64, 0), (1, 0, 16, 64, 0), (1, 1, 4097, 64, 0), (1, 1, 16, -1, 0),
                (1, 1, 16, 64, -1), (1024, 64, 128, 1 << 22, 0)):
        assert size(*bad, ctypes.byref(n)) == INVALID
    assert size(1, 1, 16, 64, 0, None) == INVALID


@pytest.mark.gpu
def test_tree_workspace_missing(m):
    """(The size depends on the device.)  Refused before any launch; what the
    query says is enough, trees of any sizes."""
    assert m.lib.mla_decode_paged_tree(*_change(TREE, mb=99, ws=P(0))) == WORKSPACE
    assert m.lib.mla_decode_paged_tree(*_change(TREE, mb=99, n=8)) == WORKSPACE
    many = dict(B=1024, q_len=64, H=128, mb=1 << 16, stride=64)
    assert m.lib.mla_decode_paged_tree(*_change(TREE, **many)) == INVALID
    for q_len, H, split in ((6, 128, 0), (12, 64, 3), (16, 128, 0), (33, 20, 5), (64, 16, 0)):
        n = m.mla_decode_tree_workspace_size(3, q_len, H, 64 * 40, split)
        q = torch.zeros((3, q_len, H, 576), dtype=torch.bfloat16, device="cuda")
        cache = torch.zeros((40, 64, 576), dtype=torch.bfloat16, device="cuda")
        args = (q, cache, torch.arange(40, dtype=torch.int32, device="cuda").repeat(3, 1),
                torch.full((3,), 64 * 40, dtype=torch.int32, device="cuda"),
                torch.ones(q_len, dtype=torch.int64, device="cuda"))
        for lens in (None, torch.tensor([q_len, 1, 0], dtype=torch.int32, device="cuda")):
            ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
            m.mla_decode_paged_tree(*args, sm_scale=1.0, split_tiles=split, tree_lens=lens, workspace=ws)
            with pytest.raises(m.MlaError):
                m.mla_decode_paged_tree(*args, sm_scale=1.0, split_tiles=split, tree_lens=lens,
                                        workspace=ws[:n // 2].contiguous())
    assert m.mla_get_device_error() == 0
