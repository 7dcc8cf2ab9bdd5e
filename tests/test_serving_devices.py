"""Every tensor of a serving call has to lie on the device that the call is launched on.  Tensors of two devices are stood in for
by host tensors that say which device they are on, and the library by one that counts calls: nothing is launched, no GPU."""
import types

import pytest
import torch

import int4_weight_only_gemm_gb300 as w

HERE, ELSEWHERE = 0, 1


class Placed(torch.Tensor):
    """A host tensor that passes for a CUDA tensor of device `index`."""
    index = HERE

    def get_device(self):
        return self.index

    @property
    def is_cuda(self):
        return True


class Other(Placed):
    index = ELSEWHERE


def on(t, cls=Placed):
    return None if t is None else t.as_subclass(cls)


@pytest.fixture
def launched(monkeypatch):
    calls = []
    names = ("w4a16_paged_attention", "w4a16_paged_attention_ex", "w4a16_kv_write", "w4a16_kv_store", "w4a16_kv_read", "w4a16_rope")
    fake = types.SimpleNamespace(**{n: (lambda *a, n=n: calls.append(n) or 0) for n in names})
    monkeypatch.setattr(w, "load_library", lambda: fake)
    monkeypatch.setattr(w, "_current", lambda: HERE)
    return calls


T, HQ, H, D, PAGES, PAGE, B = 5, 8, 2, 64, 4, 16, 2


def attention(kind):
    bf, i32 = torch.bfloat16, torch.int32
    ct = torch.int8 if kind == "int8" else bf
    a = dict(q=torch.zeros(T, HQ, D, dtype=bf), k_cache=torch.zeros(PAGES, H, PAGE, D, dtype=ct),
             v_cache=torch.zeros(PAGES, H, PAGE, D, dtype=ct), block_table=torch.zeros(B, 3, dtype=i32),
             q_start=torch.zeros(B + 1, dtype=i32), kv_len=torch.zeros(B, dtype=i32), out=torch.zeros(T, HQ, D, dtype=bf),
             lse=torch.zeros(T, HQ), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    if kind == "int8":
        a.update(k_scale=torch.zeros(PAGES, H, PAGE), v_scale=torch.zeros(PAGES, H, PAGE))
    if kind == "tree":
        a.update(tree=torch.zeros(T, 1, dtype=i32))
    return a


@pytest.mark.parametrize("kind", ["plain", "int8", "tree"])
def test_attention_refuses_each_tensor_of_another_device(launched, kind):
    tensors = attention(kind)
    call = lambda a: w.w4a16_paged_attention(**a, max_q=3, stream=0)  # noqa: E731
    call({n: on(t) for n, t in tensors.items()})
    assert len(launched) == 1
    for name in tensors:
        with pytest.raises(ValueError, match=name):
            call({n: on(t, Other if n == name else Placed) for n, t in tensors.items()})
    with pytest.raises(ValueError):   # all of them elsewhere
        call({n: on(t, Other) for n, t in tensors.items()})
    with pytest.raises(ValueError, match="CUDA"):   # or on the host
        call(tensors)
    assert len(launched) == 1


def rows(kind):
    bf, i32 = torch.bfloat16, torch.int32
    code = torch.int8 if kind.endswith("int8") else bf
    a = dict(k=torch.zeros(T, H, D, dtype=bf), v=torch.zeros(T, H, D, dtype=bf), slot_map=torch.zeros(T, dtype=i32),
             k_cache=torch.zeros(PAGES, H, PAGE, D, dtype=code), v_cache=torch.zeros(PAGES, H, PAGE, D, dtype=code))
    if kind.endswith("int8"):
        a.update(k_scale=torch.zeros(PAGES, H, PAGE), v_scale=torch.zeros(PAGES, H, PAGE))
    if kind.startswith("rope"):
        a.update(q=torch.zeros(T, HQ, D, dtype=bf), q_out=torch.zeros(T, HQ, D, dtype=bf), positions=torch.zeros(T, dtype=i32),
                 frequencies=torch.zeros(D // 2, dtype=torch.float64))
    return a


@pytest.mark.parametrize("kind", ["write", "write int8", "rope", "rope int8", "read", "read int8"])
def test_cache_calls_refuse_each_tensor_of_another_device(launched, kind):
    tensors = rows(kind)
    function = {"write": w.w4a16_kv_write, "rope": w.w4a16_rope_kv_write, "read": w.w4a16_kv_read}[kind.split()[0]]
    call = lambda a: function(**a, stream=0)  # noqa: E731
    call({n: on(t) for n, t in tensors.items()})
    assert len(launched) == 1
    for name in tensors:
        with pytest.raises(ValueError, match=name):
            call({n: on(t, Other if n == name else Placed) for n, t in tensors.items()})
    with pytest.raises(ValueError):
        call({n: on(t, Other) for n, t in tensors.items()})
    with pytest.raises(ValueError, match="CUDA"):
        call(tensors)
    assert len(launched) == 1
