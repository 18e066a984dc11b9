"""Arguments that the window and block-scaled-cache entry points refuse on
the host, before any launch (no GPU needed)."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p
OK, INVALID, WORKSPACE = 0, 1, 3
A = P(1 << 20)                  # an aligned address that nothing reads
ODD = P((1 << 20) + 8)


@pytest.fixture(scope="module")
def L():
    import mla_latent_kv_uk_gb300 as m
    return m.lib


def _change(base, **kw):
    a = dict(base)
    a.update(kw)
    return list(a.values())


APPEND = dict(q=A, qt=64 * 4, qh=64, k=A, ks=64, c=A, cs=512, pos=A, slots=A, T=3, H=4, theta=1e4, layout=0,
              q_out=A, k_out=A, cache=A, scales=A, sb=64, nb=5, s=P(0))


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=4097), dict(nb=0), dict(nb=1 << 25), dict(layout=2), dict(theta=1.0),
    dict(theta=float("inf")), dict(theta=float("nan")), dict(sb=0), dict(sb=8), dict(sb=48), dict(sb=128),
    dict(k=P(0)), dict(c=P(0)), dict(pos=P(0)), dict(slots=P(0)), dict(cache=P(0)), dict(scales=P(0)),
    dict(q=P(0)),                                       # q_out without q_pe
    dict(q=ODD), dict(k=ODD), dict(c=ODD), dict(cache=ODD), dict(q_out=ODD), dict(k_out=ODD),
    dict(ks=60), dict(ks=56), dict(cs=516), dict(cs=504), dict(qt=260), dict(qh=68), dict(qh=56),
    dict(qt=128), dict(qt=-256), dict(ks=-64)])
def test_append(L, bad):
    assert L.mla_rope_cache_append(*_change(APPEND, **bad)) == INVALID


def test_append_no_tokens(L):
    assert L.mla_rope_cache_append(*_change(APPEND, T=0, k=P(0), c=P(0), cache=P(0))) == OK


GATHER = dict(cache=A, scales=A, sb=32, bt=A, lens=A, starts=P(0), cu=A, B=2, mb=3, nb=5, rows=7, out=A, s=P(0))


@pytest.mark.parametrize("bad", [
    dict(cache=P(0)), dict(scales=P(0)), dict(bt=P(0)), dict(lens=P(0)), dict(cu=P(0)), dict(out=P(0)),
    dict(sb=1), dict(sb=63), dict(B=0), dict(mb=0), dict(nb=0), dict(nb=1 << 25), dict(rows=-1),
    dict(cache=ODD), dict(out=ODD)])
def test_gather(L, bad):
    assert L.mla_gather_cache_scaled(*_change(GATHER, **bad)) == INVALID


def test_gather_no_rows(L):
    assert L.mla_gather_cache_scaled(*_change(GATHER, rows=0, out=P(0))) == OK


DECODE = dict(q=A, qd=0, qs=1.0, kv=A, kd=0, ks=1.0, bt=A, lens=A, B=2, q_len=1, H=16, mb=3, nb=5, sm=0.1,
              window=64, sinks=4, split=0, out=A, od=0, lse=A, ws=A, n=1 << 40, s=P(0))
BAD_DECODE = [
    dict(B=0), dict(q_len=0), dict(q_len=65), dict(H=0), dict(H=4097), dict(mb=0), dict(mb=(1 << 24) + 1),
    dict(nb=0), dict(nb=1 << 25), dict(sm=0.0), dict(sm=float("nan")), dict(sm=float("inf")),
    dict(window=-1), dict(sinks=-1), dict(split=-1), dict(q=P(0)), dict(kv=P(0)), dict(bt=P(0)),
    dict(lens=P(0)), dict(out=P(0)), dict(lse=P(0)), dict(od=1), dict(q=ODD), dict(kv=ODD), dict(out=ODD),
    dict(ws=ODD), dict(B=1 << 16, q_len=64, H=4096)]


@pytest.mark.parametrize("bad", BAD_DECODE + [
    dict(qd=1), dict(kd=1), dict(qd=2, kd=2), dict(qd=1, kd=1, qs=0.0), dict(qd=1, kd=1, ks=-1.0),
    dict(qd=1, kd=1, ks=float("nan")), dict(qd=1, kd=1, ks=2.0 ** -101), dict(qd=1, kd=1, ks=2.0 ** 121)])
def test_decode_window(L, bad):
    assert L.mla_decode_paged_window(*_change(DECODE, **bad)) == INVALID


SCALED = dict(q=A, qs=1.0, kv=A, scales=A, sb=64, bt=A, lens=A, B=2, q_len=1, H=16, mb=3, nb=5, sm=0.1, window=0,
              sinks=0, split=0, out=A, od=0, lse=A, ws=A, n=1 << 40, s=P(0))


@pytest.mark.parametrize("bad", BAD_DECODE + [dict(scales=P(0)), dict(sb=0), dict(sb=24), dict(qs=0.0)])
def test_decode_scaled(L, bad):
    assert L.mla_decode_paged_scaled(*_change(SCALED, **bad)) == INVALID


@pytest.mark.gpu
def test_decode_units_beyond_32_bits(L):
    """(The grid depends on the device.)  Refused before any launch, as its
    workspace's size is."""
    many = dict(B=1024, q_len=64, H=128, mb=1 << 16, window=0)
    assert L.mla_decode_paged_window(*_change(DECODE, **many)) == INVALID
    assert L.mla_decode_paged_scaled(*_change(SCALED, **many)) == INVALID
    n = ctypes.c_size_t(0)
    assert L.mla_decode_window_workspace_size(1024, 64, 128, 1 << 22, 0, 0, 0, ctypes.byref(n)) == INVALID
    assert L.mla_decode_window_workspace_size(1024, 64, 128, 1 << 22, 128, 0, 1, ctypes.byref(n)) == OK


@pytest.mark.gpu
def test_decode_workspace_missing(L):
    """(The size depends on the device.)  Refused before any launch."""
    assert L.mla_decode_paged_window(*_change(DECODE, mb=99, window=0, ws=P(0))) == WORKSPACE
    assert L.mla_decode_paged_window(*_change(DECODE, mb=99, window=0, n=8)) == WORKSPACE
    assert L.mla_decode_paged_scaled(*_change(SCALED, mb=99, n=8)) == WORKSPACE
    assert torch.cuda.current_device() == 0


def test_decode_workspace(L):
    n = ctypes.c_size_t(0)
    assert L.mla_decode_window_workspace_size(2, 1, 16, 64 * 99, 0, 0, 0, ctypes.byref(n)) == OK and n.value > 8
    assert L.mla_decode_window_workspace_size(2, 1, 16, 64 * 99, 64, 4, 0, ctypes.byref(n)) == OK and n.value == 0
    for bad in ((0, 1, 16, 64, 0, 0, 0), (1, 65, 16, 64, 0, 0, 0), (1, 1, 16, -1, 0, 0, 0),
                (1, 1, 16, 64, -1, 0, 0), (1, 1, 16, 64, 0, -1, 0), (1, 1, 16, 64, 0, 0, -1)):
        assert L.mla_decode_window_workspace_size(*bad, ctypes.byref(n)) == INVALID
    assert L.mla_decode_window_workspace_size(1, 1, 16, 64, 0, 0, 0, None) == INVALID
    assert L.mla_decode_window_workspace_size(1, 1, 16, 64, 8, 1, 2, ctypes.byref(n)) == OK and n.value > 0


PREFILL = dict(q=A, k=A, v=A, cu_q=A, cu_k=A, B=1, Tq=4, Nk=8, H=2, mq=4, window=16, sinks=0, sm=0.1, out=A, lse=A,
               s=P(0))


@pytest.mark.parametrize("bad", [
    dict(window=0), dict(window=-3), dict(sinks=-1), dict(B=0), dict(B=65536), dict(Tq=-1), dict(Nk=-1), dict(H=0),
    dict(H=65536), dict(mq=-1), dict(sm=0.0), dict(sm=float("nan")), dict(q=P(0)), dict(k=P(0)), dict(v=P(0)),
    dict(cu_q=P(0)), dict(cu_k=P(0)), dict(out=P(0)), dict(lse=P(0)), dict(q=ODD), dict(k=ODD), dict(v=ODD),
    dict(out=ODD)])
def test_prefill_window(L, bad):
    assert L.mla_prefill_attn_window(*_change(PREFILL, **bad)) == INVALID


def test_prefill_window_no_queries(L):
    assert L.mla_prefill_attn_window(*_change(PREFILL, Tq=0, q=P(0))) == OK


# ------------------------------------------------- the Python calls' checks
def _calls(m, dev):
    """One good set of arguments for each call, by name."""
    def z(*s, dtype=torch.int32):
        return torch.zeros(s, dtype=torch.uint8 if dtype is E4M3 else dtype, device=dev).view(dtype)

    E4M3, BF = torch.float8_e4m3fn, torch.bfloat16
    cache, scales = z(3, 64, 576, dtype=E4M3), torch.ones((3, 2), device=dev)
    table, lens = z(2, 1), z(2)
    return {
        m.mla_rope_cache_append: dict(q_pe=z(4, 2, 64, dtype=BF), k_pe=z(4, 64, dtype=BF), kv_c=z(4, 512, dtype=BF),
                                      positions=z(4), slot_mapping=z(4), kv_cache=cache, kv_scales=scales,
                                      q_out=z(4, 2, 64, dtype=BF), k_out=z(4, 64, dtype=BF)),
        m.mla_gather_cache_scaled: dict(kv_cache=cache, kv_scales=scales, block_table=table, seq_lens=lens,
                                        cu_out=z(3), total_rows=0, seq_starts=z(2), out=z(0, 576, dtype=BF)),
        m.mla_decode_paged_window: dict(q=z(2, 1, 4, 576, dtype=E4M3), kv_cache=cache, block_table=table,
                                        seq_lens=lens, sm_scale=1.0, window=0, out=z(2, 1, 4, 512, dtype=BF),
                                        lse=z(2, 1, 4, dtype=torch.float32)),
        m.mla_decode_paged_scaled: dict(q=z(2, 1, 4, 576, dtype=E4M3), kv_cache=cache, kv_scales=scales,
                                        block_table=table, seq_lens=lens, sm_scale=1.0,
                                        out=z(2, 1, 4, 512, dtype=BF), lse=z(2, 1, 4, dtype=torch.float32)),
        m.mla_prefill_attn_window: dict(q=z(4, 2, 192, dtype=BF), k=z(4, 2, 192, dtype=BF), v=z(4, 2, 128, dtype=BF),
                                        cu_q=z(2), cu_k=z(2), max_q_len=0, window=8, sm_scale=1.0,
                                        out=z(4, 2, 128, dtype=BF), lse=z(4, 2, dtype=torch.float32)),
    }


@pytest.fixture(scope="module")
def m():
    import mla_latent_kv_uk_gb300 as mod
    return mod


def test_tensors_of_the_host_and_other_things(m):
    for call, kw in _calls(m, "cpu").items():
        with pytest.raises(ValueError, match="CUDA tensor"):
            call(**kw)
        with pytest.raises(TypeError, match="must be a tensor"):
            call(**{**kw, **{k: 3 for k in ("k_pe", "kv_cache", "q") if k in kw}})
        with pytest.raises(TypeError):
            call()
    with pytest.raises(KeyError):
        m.mla_rope_cache_append(**_calls(m, "cpu")[m.mla_rope_cache_append], layout="neither")


@pytest.mark.gpu
def test_python_checks(m):
    """Every tensor in turn of another type, rank, device and stride, and of
    another length; numbers that are none."""
    for call, kw in _calls(m, "cuda").items():
        call(**kw)                              # as it stands it is taken
        for name, t in kw.items():
            if not isinstance(t, torch.Tensor):
                with pytest.raises(TypeError):
                    call(**{**kw, name: "x"})
                continue
            for bad, errors in ((t.unsqueeze(0), ValueError), (t.cpu(), ValueError),
                                (torch.zeros(t.shape, dtype=torch.float64, device="cuda"), TypeError),
                                ([1], TypeError)):
                with pytest.raises(errors):
                    call(**{**kw, name: bad})
            if t.numel() > 1:
                wide = torch.zeros((*t.shape, 2), dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype,
                                   device="cuda").view(t.dtype)[..., 0]
                with pytest.raises(ValueError):
                    call(**{**kw, name: wide})
            if t.numel() and (name != "kv_cache" or "kv_scales" in kw):    # (else any number of blocks will do)
                with pytest.raises((ValueError, TypeError)):
                    call(**{**kw, name: t[:-1]})
        with pytest.raises(ValueError):
            call(**{**kw, **({"total_rows": 2 ** 40} if "total_rows" in kw else
                             {"max_q_len": -2 ** 40} if "max_q_len" in kw else
                             {"split_tiles": 2 ** 31} if "sm_scale" in kw else {"kv_scales": kw["kv_scales"][:, :0]})})
    assert m.mla_get_device_error() in (0, 1)   # (the tables' zeros are block 0)


@pytest.mark.gpu
def test_status_becomes_the_librarys_error(m):
    kw = _calls(m, "cuda")[m.mla_prefill_attn_window]
    with pytest.raises(m.MlaError) as e:
        m.mla_prefill_attn_window(**{**kw, "window": 0})
    assert e.value.status == INVALID and "mla_prefill_attn_window" in str(e.value)
    kw = _calls(m, "cuda")[m.mla_decode_paged_window]
    with pytest.raises(m.MlaError) as e:
        m.mla_decode_paged_window(**{**kw, "split_tiles": 1, "workspace": torch.zeros(8, dtype=torch.uint8, device="cuda")})
    assert e.value.status == WORKSPACE
