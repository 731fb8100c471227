"""Stand-ins for streams and the library, to see on the CPU whose memory a call allocates."""
import torch


class Streams:
    """Stand-ins for the device side of the binding: calls return 0, and every torch.empty notes the stream whose
    memory it would come from."""

    def __init__(self, A, monkeypatch):
        self.now, self.made, self.recorded = "current", [], []
        fake = self

        class Within:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                fake.before, fake.now = fake.now, self.stream

            def __exit__(self, *_):
                fake.now = fake.before

        real = {name: getattr(torch, name) for name in ("empty", "empty_like")}

        def making(name):
            def make(*args, **kw):
                x = real[name](*args, **kw)
                fake.made.append((fake.now, x.data_ptr()))
                return x
            return make

        class Library:
            def __getattr__(self, name):
                return lambda *args: 4096 if name.endswith("_size") else 0

        monkeypatch.setattr(A, "_lib", Library())
        monkeypatch.setattr(A, "_raw_stream", lambda stream, index: 0)
        monkeypatch.setattr(A, "_stream", lambda stream: None)
        monkeypatch.setattr(torch.cuda, "stream", Within)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: "current")
        monkeypatch.setattr(torch.Tensor, "record_stream", lambda x, s: fake.recorded.append((s, x.data_ptr())),
                            raising=False)
        for name in real:
            monkeypatch.setattr(torch, name, making(name))

    def check(self, returned):
        """All memory was the given stream's, and the caller's stream is on record for what it gets."""
        assert self.made and all(stream == "given" for stream, _ in self.made), self.made
        for x in returned:
            assert ("current", x.data_ptr()) in self.recorded
