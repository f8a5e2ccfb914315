"""What a build prints is what it runs (no compiler is started)."""
import os

from moe_expert_load_ultraep_amd import _build


def test_build_prints_the_commands_it_runs(monkeypatch, tmp_path, capsys):
    ran = []

    class Done:
        returncode = 0

    def run(cmd, **kw):
        ran.append(" ".join(cmd))
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done

    monkeypatch.setattr(_build, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build.subprocess, "run", run)
    assert _build.build(verbose=True) == str(tmp_path / "lib.so") and os.path.exists(tmp_path / "lib.so")
    printed = capsys.readouterr().out.splitlines()
    assert sorted(printed) == sorted(ran) and len(ran) == len(_build.SOURCES) + 1
    assert sum(" -c " in c for c in ran) == len(_build.SOURCES) and " -shared " in ran[-1]
    for s in _build.SOURCES:
        assert sum(os.path.join(_build.CSRC, s) in c for c in ran) == 1
    _build.build()
    assert capsys.readouterr().out == ""
