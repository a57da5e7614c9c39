"""Host: the Python binding refuses every tensor (and stream) that is not the current device's, before anything is called.
Stand-ins for tensors on GPUs, and for the library, so that no GPU is needed."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
import dflash2_block_drafter_gb300 as d  # noqa: E402


class On(torch.Tensor):
    """A host tensor that says it lies on cuda:`place`."""
    place = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.place


def _on(t, place=0):
    t = t.as_subclass(On)
    t.place = place
    return t


class _Library:
    """Takes every call: sizes of workspaces are 256, the rest returns 0."""
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_bytes"):
                return 256
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    lib = _Library()
    monkeypatch.setattr(d, "library", lambda: lib)
    monkeypatch.setattr(d, "_current_device", lambda: 0)
    d.dflash2_logits_topk_workspace_bytes.cache_clear()
    yield lib
    d.dflash2_logits_topk_workspace_bytes.cache_clear()


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def _f32(*s):
    return torch.zeros(s)


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


B, G, HQ, HKV, D, PAGE, H, F, K, V, R = 2, 3, 4, 2, 64, 16, 64, 128, 16, 64, 32
CACHE = lambda: _u8(5, HKV, 2, 1, 16 * (D // 2 + D // 64 * 4))
ATT = dict(q=_bf(B, G, HQ, D), cache=CACHE(), page_table=_i32(B, 4), ctx_len=_i32(B), k_new=_bf(B, G, HKV, D),
           v_new=_bf(B, G, HKV, D), out=_bf(B, G, HQ, D), workspace=_u8(256))
SITE = dict(w_kp=_bf(4 * H // 16, H), workspace=_u8(256))
PROJ = dict(w=_i32(F, H // 8), w_scales=_bf(H // 64, F), w_biases=_bf(H // 64, F), out=_bf(B * G, F), workspace=_u8(256))
HEAD = dict(h=_bf(6, H), w_proj=_bf(R, H), cand=_i32(6, K), unary=_f32(6, K), z=_f32(6, R), logits=_f32(6, V))
BOOKS = dict(pred_book=_bf(V, R), succ_book=_bf(V, R), anchors=_i32(B))
EDGES = dict(BOOKS, cand=_i32(B, 4, K), unary=_f32(B, 4, K), z=_f32(B, 4, R), S=_f32(B, 4, K, K), path=_i32(B, 4))
CALLS = [
    ("dflash2_kv4_plan", dict(page_size=PAGE, num_pages=9, rows=8),
     dict(ctx_len=_i32(B), change=_i32(B), page_table=_i32(B, 4), free_pages=_i32(9), free_state=_i32(2), place=_i32(B, G),
          ctx_out=_i32(B), state_out=_i32(2), offsets=_i32(B + 1), slots=torch.zeros(B, G, dtype=torch.int64),
          positions=_i32(B, G))),
    ("dflash2_kv4_attention", dict(page_size=PAGE, scale=1.0), ATT),
    ("dflash2_kv4_attention_tree", dict(page_size=PAGE, scale=1.0), dict(ATT, parents=_i32(B, G))),
    ("dflash2_kv4_append", dict(page_size=PAGE),
     dict(k=_bf(7, HKV, D), v=_bf(7, HKV, D), slots=torch.zeros(7, dtype=torch.int64), cache=CACHE())),
    ("dflash2_kv4_read", dict(head_dim=D, page_size=PAGE),
     dict(cache=CACHE(), slots=torch.zeros(7, dtype=torch.int64), k=_bf(7, HKV, D), v=_bf(7, HKV, D))),
    ("dflash2_logits_topk", dict(K=K, requests=B),
     dict(logits=_f32(6, V), row_offsets=_i32(B + 1), history=_i32(B, 5), prompt_len=_i32(B), history_len=_i32(B),
          repetition=_f32(B), frequency=_f32(B), presence=_f32(B), tokens=_i32(6), parents=_i32(6), bias_ids=_i32(B, 2),
          bias=_f32(B, 2), mask=_i32(6, V // 32), cand=_i32(6, K), unary=_f32(6, K), out=_f32(6, V), workspace=_u8(512))),
    ("dflash2_gated_ffn", dict(),
     dict(x=_bf(6, H), w_gate=_bf(F, H), w_up=_bf(F, H), out=_bf(6, F), pre=_i32(6, F), workspace=_u8(256))),
    ("dflash2_gated_ffn_backward", dict(),
     dict(dh=_bf(6, F), pre=_i32(6, F), x=_bf(6, H), w_gate=_bf(F, H), w_up=_bf(F, H), dx=_bf(6, H), dw_gate=_bf(F, H),
          dw_up=_bf(F, H), workspace=_u8(256))),
    ("dflash2_proj", dict(), dict(PROJ, a=_bf(B * G, H))),
    ("dflash2_proj_conv_in", dict(G=G, group_size=16),
     dict(PROJ, n=_bf(B * G, H), d0=_f32(2, H // 16, B * G), base=_f32(2, 2, H))),
    ("dflash2_proj_conv_out", dict(G=G, group_size=16),
     dict(PROJ, a=_bf(B * G, H), coef1=_bf(B * G, 2, F // 16), base=_f32(2, 2, F), residual=_bf(B * G, F))),
    ("dflash2_conv_prepare", dict(eps=1e-6, group_size=16),
     dict(SITE, x=_bf(B, G, H), norm_w=_bf(H), base=_f32(2, 2, H), out=_bf(B, G, H), coef1=_bf(B, G, 2, H // 16),
          d_full=_f32(B * G, 4 * H // 16))),
    ("dflash2_conv_coefficients", dict(eps=1e-6, group_size=16),
     dict(SITE, x=_bf(B, G, H), norm_w=_bf(H), n_out=_bf(B * G, H), d0=_f32(2, H // 16, B * G), coef1=_bf(B * G, 2, H // 16))),
    ("dflash2_conv_finish", dict(group_size=16),
     dict(y=_bf(B, G, H), coef1=_bf(B, G, 2, H // 16), base=_f32(2, 2, H), residual=_bf(B, G, H), out=_bf(B, G, H),
          next_norm_w=_bf(H), next_n=_bf(B, G, H))),
    ("dflash2_conv_finish_ragged", dict(group_size=16, m_rows=4),
     dict(y=_bf(B, G, H), coef1=_bf(B, G, 2, H // 16), base=_f32(2, 2, H), row_offsets=_i32(B + 1), next_norm_w=_bf(H),
          residual=_bf(B, G, H), out=_bf(B, G, H), next_n=_bf(4, H))),
    ("dflash2_head_topk", dict(K=K), dict(HEAD, w_head=_bf(V, H), bias=_f32(V), workspace=_u8(256))),
    ("dflash2_head_topk_noalloc", dict(K=K), dict(HEAD, w_head=_bf(V, H), bias=_f32(V))),
    ("dflash2_head_topk_vocab", dict(K=K),
     dict(HEAD, w_listed=_bf(V, H), vocab_ids=_i32(V), bias_listed=_f32(V), workspace=_u8(256))),
    ("dflash2_score_edges", dict(), EDGES),
    ("dflash2_score_edges_depths", dict(), dict(EDGES, depths=_i32(B))),
    ("dflash2_score_edges_ragged", dict(steps=4),
     dict(BOOKS, cand=_i32(6, K), unary=_f32(6, K), z=_f32(6, R), row_offsets=_i32(B + 1), S=_f32(6, K, K), path=_i32(B, 4))),
    ("dflash2_select_path", dict(), dict(S=_f32(B, 4, K, K), cand=_i32(B, 4, K), path=_i32(B, 4))),
    ("dflash2_select_path_depths", dict(),
     dict(S=_f32(B, 4, K, K), cand=_i32(B, 4, K), depths=_i32(B), path=_i32(B, 4))),
]


@pytest.mark.parametrize("name,plain,tensors", CALLS, ids=[c[0] for c in CALLS])
def test_each_tensor_of_another_device_is_refused(fake, name, plain, tensors):
    call = getattr(d, name)
    here = {k: _on(t) for k, t in tensors.items()}
    call(**plain, **here, stream=0)
    assert fake.calls == [name]
    for k, t in tensors.items():
        with pytest.raises(ValueError, match=rf"{k} is on cuda:1, the current device is cuda:0"):
            call(**plain, **dict(here, **{k: _on(t, 1)}), stream=0)
    assert fake.calls == [name]


def test_a_stream_of_another_device_is_refused(fake):
    class Stream:
        cuda_stream, device_index = 0, 1

    t = {k: _on(x) for k, x in dict(S=_f32(B, 4, K, K), cand=_i32(B, 4, K), path=_i32(B, 4)).items()}
    with pytest.raises(ValueError, match="stream is of cuda:1"):
        d.dflash2_select_path(**t, stream=Stream())
    assert fake.calls == []
    Stream.device_index = 0
    d.dflash2_select_path(**t, stream=Stream())
    assert fake.calls == ["dflash2_select_path"]
    assert isinstance(d._stream(Stream()), ctypes.c_void_p)
