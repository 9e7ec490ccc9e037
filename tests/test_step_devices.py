"""The binding's calls of a step over long contexts refuse every tensor that is not on the current device before the
library is called: its kernels would read the address as their own memory.  No GPU needed: the tensors below lie on the
CPU, which is made the current device, and one of them says that it lies elsewhere."""
import pytest

from dspark_markov_draft_anchor_gb300 import binding

torch = pytest.importorskip("torch")

I = torch.int32  # noqa: E741
ROWS, HEADS, DIM, PAGES = 3, 2, 64, 4


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 7


class Library:
    """Takes every call and says that all is well."""

    def __getattr__(self, name):
        return lambda *a: 1 if name.endswith("bytes") else 0


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def tensors():
    """Every tensor of the calls by its name."""
    bf16, rows = torch.bfloat16, (ROWS, HEADS, DIM)
    return dict(data=z(PAGES, binding.kv4_page_bytes(16, HEADS, DIM), dtype=torch.uint8), k_scale=z(HEADS), v_scale=z(HEADS),
                row_start=z(2, dtype=I), lens=z(1, dtype=I), table=z(1, PAGES, dtype=I), slots=z(1, dtype=I),
                cos=z(9, 32), sin=z(9, 32), positions=z(ROWS, dtype=I), k=z(*rows, dtype=bf16), v=z(*rows, dtype=bf16),
                q=z(*rows, dtype=bf16), out=z(*rows, dtype=bf16), lse=z(ROWS, HEADS),
                bounds=z(PAGES, binding.kv4_bounds_bytes(HEADS, DIM), dtype=torch.uint8),
                pages=z(ROWS, HEADS, 2, dtype=I), kept=z(ROWS, dtype=I), workspace=z(4096, dtype=torch.uint8),
                counts=z(2, 40, dtype=I), marks=z(2, 2, 2, dtype=I), tokens=z(2, 5, dtype=torch.int64), held=z(2, dtype=I),
                logits=z(4, 40), y=z(4, 40), draft=z(2, 1, dtype=torch.int64), repetition=z(2), frequency=z(2),
                presence=z(2), start=z(3, dtype=I), ids=z(5, dtype=I), values=z(5), mask=z(4, 2, dtype=I),
                mask_rows=z(4, dtype=I), at=z(2, dtype=I))


CACHE, BATCH = ("data", "k_scale", "v_scale"), ("row_start", "lens", "table", "slots")
READ = dict(
    append=(*CACHE, *BATCH, "cos", "sin", "positions", "k", "v"),
    rotate=(*CACHE, *BATCH, "cos", "sin", "positions", "k", "v", "q", "out"),
    bound=(*CACHE, *BATCH, "bounds"),
    select=(*CACHE, *BATCH, "bounds", "q", "pages", "kept", "workspace"),
    attend=(*CACHE, "pages", "kept", "q", "out", "lse", "workspace"),
    count=("counts", "marks", "tokens", "held", "at"),
    adjust=("counts", "marks", "logits", "y", "at", "draft", "repetition", "frequency", "presence", "start", "ids", "values",
            "mask", "mask_rows"),
)


def call(name, t):
    cache = binding.Kv4Cache(t["data"], 16, HEADS, DIM, k_scale=t["k_scale"], v_scale=t["v_scale"])
    batch = binding.Kv4Batch(t["row_start"], t["lens"], t["table"], total_rows=ROWS, max_rows=ROWS, slots=t["slots"])
    rotation = binding.Kv4Rotation(t["cos"], t["sin"], positions=t["positions"])
    selection = binding.Kv4Selection(t["pages"], t["kept"])
    table = binding.TokenTable(t["counts"], t["marks"])
    if name == "append":
        binding.dspark_kv4_append_rotated(cache, batch, rotation, t["k"], t["v"], stream=1)
    elif name == "rotate":
        binding.dspark_kv4_append_rotated(cache, batch, rotation, t["k"], t["v"], t["q"], t["out"], stream=1)
    elif name == "bound":
        binding.dspark_kv4_bound_pages(cache, batch, t["bounds"], stream=1)
    elif name == "select":
        binding.dspark_kv4_select(cache, batch, t["bounds"], t["q"], selection, t["workspace"], stream=1)
    elif name == "attend":
        binding.dspark_kv4_attention_selected(cache, selection, t["q"], t["out"], 1.0, t["workspace"], lse=t["lse"], stream=1)
    elif name == "count":
        binding.dspark_tokens_count(table, t["tokens"], t["held"], slots=t["at"], stream=1)
    else:
        binding.dspark_logits_adjust(table, t["logits"], t["y"], drafts=1, slots=t["at"], draft=t["draft"],
                                     repetition=t["repetition"], frequency=t["frequency"], presence=t["presence"],
                                     bias=(t["start"], t["ids"], t["values"]), mask=t["mask"], mask_rows=t["mask_rows"],
                                     stream=1)


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: -1)


@pytest.mark.parametrize("name", READ)
def test_tensors_on_the_current_device_are_taken(name, monkeypatch):
    monkeypatch.setattr(binding, "load", Library)
    call(name, tensors())


@pytest.mark.parametrize("name,which", [(name, which) for name, read in READ.items() for which in read])
def test_a_tensor_on_another_device_is_refused(name, which, monkeypatch):
    monkeypatch.setattr(binding, "load", lambda: pytest.fail("the library was called"))
    t = tensors()
    t[which] = t[which].as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="current device"):
        call(name, t)


@pytest.mark.parametrize("name", ["select", "attend"])
def test_a_workspace_with_bytes_of_others_between_is_refused(name, monkeypatch):
    monkeypatch.setattr(binding, "load", lambda: pytest.fail("the library was called"))
    for spread in (z(8192, dtype=torch.uint8)[::2], z(64, 128, dtype=torch.uint8)[:, :64], z(64, 1, dtype=torch.uint8).expand(64, 64)):
        with pytest.raises(ValueError, match="workspace"):
            call(name, dict(tensors(), workspace=spread))


def test_the_whole_caches_attention_refuses_such_a_workspace_too(monkeypatch):
    monkeypatch.setattr(binding, "load", lambda: pytest.fail("the library was called"))
    t = tensors()
    cache = binding.Kv4Cache(t["data"], 16, HEADS, DIM)
    batch = binding.Kv4Batch(t["row_start"], t["lens"], t["table"], total_rows=ROWS, max_rows=ROWS)
    with pytest.raises(ValueError, match="workspace"):
        binding.dspark_kv4_attention(cache, batch, t["q"], t["out"], 1.0, z(8192, dtype=torch.uint8)[::2], stream=1)
