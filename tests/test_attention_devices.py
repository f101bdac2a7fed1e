"""The attention operators' tensors lie on one device, and that is the current one:
the library launches there, with pointers that it cannot look into.  Checked with
stand-ins for tensors, which name their device and have no memory."""
import pytest
import torch

import swiglu_mlp_group_gb300 as ck

BF16, I32, I64, F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32


class Stub:
    """What the binding asks of a tensor: contiguous, of a shape and type, on a device (-1: the host)."""

    def __init__(self, shape, dtype=BF16, dev=0):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        self.is_cuda = dev >= 0
        self.device = torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")

    def get_device(self):
        return self.dev

    def stride(self):
        st, n = [], 1
        for d in reversed(self.shape):
            st.insert(0, n)
            n *= d
        return tuple(st)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x10000


class FakeLib:
    """Stands for the library: every entry point records its name and succeeds."""

    def __init__(self, calls):
        self.calls = calls

    def __getattr__(self, name):
        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def calls(monkeypatch):
    """The entry points that were called, with device 0 current."""
    made = []
    monkeypatch.setattr(ck, "lib", lambda: FakeLib(made))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return made


def norm_rope(**over):
    a = dict(q=Stub((3, 4, 64)), k=Stub((3, 2, 64)), cos_sin=Stub((9, 64), F32), positions=Stub((3,), I32),
             wq=Stub((64,)), wk=Stub((64,)), q_out=Stub((3, 4, 64)), k_out=Stub((3, 2, 64)))
    return ck.qk_norm_rope(**{**a, **over})


def append(**over):
    a = dict(k=Stub((3, 2, 64)), v=Stub((3, 2, 64)), k_cache=Stub((5, 2, 16, 64)), v_cache=Stub((5, 2, 16, 64)),
             slots=Stub((3,), I64), cos_sin=Stub((9, 64), F32), positions=Stub((3,), I32), wk=Stub((64,)))
    return ck.kv_append(**{**a, **over})


def prefix(**over):
    a = dict(q=Stub((2, 1, 4, 64)), k_cache=Stub((5, 2, 16, 64)), v_cache=Stub((5, 2, 16, 64)),
             prefix_pages=Stub((2,), I32), prefix_len=20, block_table=Stub((2, 2), I32), seq_lens=Stub((2,), I32),
             max_seq_len=30, out=Stub((2, 1, 4, 64)), workspace=Stub((1 << 20,), torch.uint8))
    return ck.prefix_attention(**{**a, **over})


def cross(**over):
    a = dict(q=Stub((2, 1, 4, 64)), k=Stub((2, 7, 2, 64)), v=Stub((2, 7, 2, 64)), kv_lens=Stub((2,), I32),
             out=Stub((2, 1, 4, 64)), workspace=Stub((1 << 20,), torch.uint8))
    return ck.cross_attention(**{**a, **over})


CALLS = [(norm_rope, ["q", "k", "cos_sin", "positions", "wq", "wk", "q_out", "k_out"]),
         (append, ["k", "v", "k_cache", "v_cache", "slots", "cos_sin", "positions", "wk"]),
         (prefix, ["q", "k_cache", "v_cache", "prefix_pages", "block_table", "seq_lens", "out", "workspace"]),
         (cross, ["q", "k", "v", "kv_lens", "out", "workspace"])]


def elsewhere(call, names, dev, monkeypatch):
    """The call's arguments of these names on another device."""
    import inspect
    base = {}

    def grab(*args, **kw):
        base.update(kw)
    target = {norm_rope: "qk_norm_rope", append: "kv_append", prefix: "prefix_attention", cross: "cross_attention"}[call]
    with monkeypatch.context() as m:
        m.setattr(ck, target, grab)
        call()
    assert inspect.signature(getattr(ck, target)).parameters.keys() >= base.keys()
    return {n: Stub(base[n].shape, base[n].dtype, dev) for n in names}


@pytest.mark.parametrize("call", [c for c, _ in CALLS])
def test_one_device_is_accepted(call, calls):
    call()
    assert len(calls) == 1


@pytest.mark.parametrize("dev", [-1, 1])
@pytest.mark.parametrize("call,name", [(c, n) for c, ns in CALLS for n in ns])
def test_one_tensor_elsewhere(call, name, dev, calls, monkeypatch):
    with pytest.raises(ValueError):
        call(**elsewhere(call, [name], dev, monkeypatch))
    assert not calls


@pytest.mark.parametrize("call,names", CALLS)
def test_all_on_a_device_that_is_not_current(call, names, calls, monkeypatch):
    with pytest.raises(ValueError):
        call(**elsewhere(call, names, 1, monkeypatch))
    assert not calls
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    call(**elsewhere(call, names, 1, monkeypatch))
    assert len(calls) == 1
