"""The step calls' two ways through the binding (the extension module, and the checks in Python that it leaves
odd arguments to) give the same results and the same refusals; and a whole step of them together."""

import numpy as np
import pytest
import torch

import attention_fa2_attn_gb300 as fa
import fa_inputs as fi
import oracle
from attention_fa2_attn_gb300 import _lib, api
from parity import compare

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


class _Odd:
    """An extension module that leaves everything to the checks in Python."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture(params=["extension", "python"])
def way(request, monkeypatch):
    if request.param == "python":
        monkeypatch.setattr(api, "fast", lambda: _Odd())
    return request.param


def _state():
    B, Hq, Hkv, T, d, mp = 3, 6, 2, 5, 64, 9
    g = torch.Generator().manual_seed(1)
    fused = fi.randn((B, T, Hq + 2 * Hkv, d), 2).to(DEV)
    q, k, v = (x.transpose(1, 2) for x in fused.split([Hq, Hkv, Hkv], dim=2))
    P = B * mp + 1
    return dict(B=B, T=T, q=q, k=k, v=v, kp=fi.randn((P, 16, Hkv, d), 3).to(DEV), vp=fi.randn((P, 16, Hkv, d), 4).to(DEV),
                cached=_i32([100, 0, 37]), new=_i32([5, 4, 2]), free=_i32(torch.randperm(P - 1, generator=g) + 1),
                table=_i32(np.zeros((B, mp))), parents=_i32([[-1, 0, 0, 1, 2]] * B), inv=fa.fa_rope_inv_freq(32)[0])


def _step(s):
    """One step that verifies drafts: plan, tree mask, rotate and append, attention."""
    # the cached tokens' pages, as an earlier plan left them
    fa.fa_paged_plan(torch.zeros_like(s["cached"]), s["cached"], s["free"], s["table"], 128)
    used = int((-(-s["cached"].cpu() // 16)).sum())
    seqlens, slots, _, need = fa.fa_paged_plan(s["cached"], s["new"], s["free"][used:].contiguous(), s["table"], s["T"])
    mask, positions = fa.fa_tree_mask(s["parents"], seqlens, s["new"])
    qr = fa.fa_rope_append_paged(s["q"], s["k"], s["v"], positions, slots, s["inv"], s["kp"], s["vp"])
    o, lse = fa.fa_tree_decode_paged(qr, s["kp"], s["vp"], s["table"], seqlens, mask, s["new"])
    return dict(seqlens=seqlens, slots=slots, need=need, mask=mask, positions=positions, qr=qr, o=o, lse=lse)


def test_a_whole_step(way):
    s = _state()
    s["vp"].mul_(0.25), s["v"].mul_(0.25)
    got = _step(s)
    assert fa.fa_get_last_device_error()[0] == 0
    # the same from the oracles, the rotated rows and pages rebuilt from the inputs
    t = _state()
    t["vp"].mul_(0.25), t["v"].mul_(0.25)
    free = t["free"].cpu().numpy()
    table, *_, used, ok = oracle.paged_plan(np.zeros(3), t["cached"], free, t["table"], 128)
    table, seqlens, slots, _, need, ok2 = oracle.paged_plan(t["cached"], t["new"], free[used:], table, t["T"])
    assert ok and ok2 and np.array_equal(s["table"].cpu().numpy(), table) and int(got["need"]) == need
    assert np.array_equal(got["slots"].cpu().numpy(), slots) and np.array_equal(got["seqlens"].cpu().numpy(), seqlens)
    positions = np.zeros((3, 5), np.int64)
    words = np.zeros((3, 5, 1), np.uint32)
    for b, n in enumerate((5, 4, 2)):
        sees, depth = oracle.tree_sees([-1, 0, 0, 1, 2], n)
        words[b], positions[b, :n] = oracle.pack_words(sees, 5), seqlens[b] - n + depth
    assert np.array_equal(got["positions"].cpu().numpy(), positions)
    assert np.array_equal(got["mask"].cpu().numpy().view(np.uint32), words)
    qr = torch.from_numpy(oracle.rope(t["q"], positions, t["inv"])).bfloat16()
    kr = torch.from_numpy(oracle.rope(t["k"], positions, t["inv"])).bfloat16()
    assert (got["qr"].cpu().float() - qr.float()).abs().max() <= 2.0 ** -7 * qr.float().abs().max()  # a rounding apart at most
    kp, vp = t["kp"].cpu(), t["vp"].cpu()
    for b in range(3):
        for i in range(5):
            if slots[b, i] >= 0:
                kp.view(-1, 2, 64)[slots[b, i]] = kr[b, :, i]
                vp.view(-1, 2, 64)[slots[b, i]] = t["v"][b, :, i].cpu()
    assert torch.equal(s["vp"].cpu(), vp)
    assert (s["kp"].cpu().float() - kp.float()).abs().max() <= 2.0 ** -7 * kr.float().abs().max()
    o_ref, lse_ref = oracle.tree_attention(got["qr"], s["kp"], s["vp"], table, seqlens, words.view(np.int32), [5, 4, 2])
    compare(got["o"], got["lse"], o_ref, lse_ref)


def test_both_ways_agree(monkeypatch):
    a = _step(s1 := _state())
    monkeypatch.setattr(api, "fast", lambda: _Odd())
    b = _step(s2 := _state())
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert torch.equal(s1["kp"], s2["kp"]) and torch.equal(s1["vp"], s2["vp"]) and torch.equal(s1["table"], s2["table"])


def test_the_extension_takes_the_plain_calls(monkeypatch):
    # the checks in Python end in ctypes calls: none is made for a step's arguments
    s = _state()
    _lib.fast()
    want = _step(_state())
    real = _lib.lib()

    class NoCalls:
        def __getattr__(self, name):
            assert name.startswith(("fa_get", "fa_tree_workspace")), name
            return getattr(real, name)

    monkeypatch.setattr(api, "lib", lambda: NoCalls())
    got = _step(s)
    assert all(torch.equal(got[n], want[n]) for n in got)
    out = (torch.empty_like(s["q"]), torch.empty_like(s["k"]))
    pos = got["positions"]
    r = fa.fa_rope(s["q"], s["k"], pos, s["inv"], q_out=out[0], k_out=out[1])
    assert r[0] is out[0] or r[0].data_ptr() == out[0].data_ptr()
    fa.fa_rope_append_paged(s["q"], s["k"], s["v"], pos, got["slots"], s["inv"], s["kp"], s["vp"], q_out=out[0])


def _wrong(s):
    """(call, what is wrong) for each argument of each call."""
    B, T = s["B"], s["T"]
    i64 = s["new"].long()
    plan = dict(cached_lens=s["cached"], new_lens=s["new"], free_pages=s["free"], block_table=s["table"], T=T)
    for change in ({"cached_lens": i64}, {"cached_lens": s["new"][:2]}, {"new_lens": _i32([1, 2, 3, 4])}, {"free_pages": s["table"]},
                   {"block_table": s["table"].t()}, {"block_table": s["new"]}, {"T": 0}, {"T": -3}, {"new_lens": s["new"].cpu()},
                   {"slots": s["table"]}, {"positions": torch.empty(B, T, dtype=torch.int64, device=DEV)},
                   {"cached_lens": _i32([1, 9, 2, 9, 3, 9])[::2]}):
        yield lambda c=change: fa.fa_paged_plan(**dict(plan, **c)), change
    seqlens = s["cached"] + s["new"]
    for change in ({"parents": s["new"]}, {"parents": s["parents"].long()}, {"seqlens": s["new"][:2]}, {"tree_lens": i64},
                   {"mask": s["table"]}, {"parents": s["parents"].cpu()}):
        yield lambda c=change: fa.fa_tree_mask(**dict(dict(parents=s["parents"], seqlens=seqlens), **c)), change
    pos = _i32(np.zeros((B, T)))
    q, k, v = s["q"], s["k"], s["v"]
    rope = dict(q=q, k=k, positions=pos, inv_freq=s["inv"])
    rope_wrong = [{"q": q.half()}, {"q": q[0]}, {"q": q.transpose(2, 3)}, {"k": k.float()}, {"k": k[:2]}, {"positions": pos.long()},
                  {"positions": pos[:2]}, {"inv_freq": s["inv"].float()}, {"inv_freq": s["inv"][None]}, {"q": q.cpu()},
                  {"inv_freq": s["inv"].cpu()}, {"q_out": q.float()}, {"q_out": k}, {"k_out": k[:, :1].expand_as(k)},
                  {"q_out": torch.empty(3, 6, 5, 128, dtype=q.dtype, device=DEV)[..., ::2]},
                  {"k": None, "k_out": torch.empty_like(k)}]
    for change in rope_wrong:
        yield lambda c=change: fa.fa_rope(**dict(rope, **c)), change
    app = dict(q=q, k=k, v=v, positions=pos, slots=pos, inv_freq=s["inv"], k_pages=s["kp"], v_pages=s["vp"])
    for change in ({"q": q.float()}, {"k": q}, {"v": v[:2]}, {"positions": pos[0]}, {"slots": pos.long()}, {"slots": pos[:2]},
                   {"k_pages": s["kp"].float()}, {"v_pages": s["vp"][:3]}, {"k_pages": s["kp"].transpose(1, 2)}, {"q_out": k},
                   {"k_pages": s["kp"].cpu()}):
        yield lambda c=change: fa.fa_rope_append_paged(**dict(app, **c)), change
    mask = _i32(np.zeros((B, T, 1)))
    tree = dict(q=q.contiguous(), k_pages=s["kp"], v_pages=s["vp"], block_table=s["table"], seqlens=seqlens, tree_mask=mask)
    for change in ({"q": q}, {"q": q.float()}, {"k_pages": s["kp"][..., :32]}, {"v_pages": s["vp"][:3]}, {"block_table": s["table"][:2]},
                   {"seqlens": i64}, {"seqlens": seqlens[:2]}, {"tree_mask": mask[:2]}, {"tree_mask": mask.long()},
                   {"tree_mask": _i32(np.zeros((T, 2)))}, {"tree_lens": i64}, {"tree_lens": s["new"][:1]}, {"seqlens": seqlens.cpu()},
                   {"out": q.float()}, {"lse": torch.empty(B, 6, T, dtype=torch.float64, device=DEV)},
                   {"block_table": torch.zeros(B, 65536, dtype=torch.int32, device=DEV),
                    "workspace": torch.empty(16, dtype=torch.uint8, device=DEV)}):
        yield lambda c=change: fa.fa_tree_decode_paged(**dict(tree, **c)), change


def test_refusals_by_name(way):
    for call, change in _wrong(_state()):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"not refused: {list(change)}")
    torch.cuda.synchronize()
    assert fa.fa_get_last_device_error()[0] == 0


def test_unsupported_sizes_are_errors_of_the_library(way):
    s = _state()
    with pytest.raises(fa.FAError) as e:
        fa.fa_rope(s["q"], s["k"], _i32(np.zeros((3, 5))), torch.zeros(40, dtype=torch.float64, device=DEV))  # 80 of 64 rotated
    assert e.value.status == _lib.FA_ERR_INVALID_ARG
    kp = fi.randn((4, 16, 2, 96), 5).to(DEV)
    with pytest.raises(fa.FAError) as e:
        fa.fa_tree_decode_paged(fi.randn((1, 2, 1, 96), 6).to(DEV), kp, kp, _i32([[0]]), _i32([3]), _i32([[1]]))
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED
    with pytest.raises(fa.FAError) as e:
        fa.fa_tree_mask(_i32(np.zeros((1, 9000)) - 1), _i32([9000]))
    assert e.value.status == _lib.FA_ERR_UNSUPPORTED


def test_integer_scale_and_flags(way):
    # whole numbers where floats and truth values are meant go the checks' way and mean the same
    s = _state()
    a = fa.fa_rope(s["q"], s["k"], _i32(np.ones((3, 5))), s["inv"], interleaved=1, mscale=2)
    b = fa.fa_rope(s["q"], s["k"], _i32(np.ones((3, 5))), s["inv"], interleaved=True, mscale=2.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_inputs_of_another_stream(way):
    # the call runs on the current stream, after what that stream waits for
    s = _state()
    pos = _i32(np.zeros((3, 5)))
    want = fa.fa_rope(s["q"], s["k"], pos + 3, s["inv"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        big = torch.randn(1 << 26, device=DEV)
        for _ in range(5):
            big = big * 1.0001
        pos.copy_(torch.full_like(pos, 3))
        got = fa.fa_rope(s["q"], s["k"], pos, s["inv"])
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
