"""A library of another version, or without some entry points, is named as such when it is loaded."""
import subprocess

import pytest

pytest.importorskip("torch")

import activation_sparse_predict_amd as pi  # noqa: E402


def load(tmp_path, monkeypatch, version, names):
    src = "\n".join(f"int {n}(void) {{ return {version if n == 'pi_abi_version' else 0}; }}" for n in names)
    (tmp_path / "lib.c").write_text(src + "\n")
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "lib.c"), "-o", str(tmp_path / "libpi.so")], check=True)
    monkeypatch.setattr(pi, "LIB_PATH", str(tmp_path / "libpi.so"))
    monkeypatch.setattr(pi, "_lib", None)
    with pytest.raises(RuntimeError) as e:
        pi.lib()
    assert pi._lib is None and "rebuild" in str(e.value)
    return str(e.value)


def test_an_older_version_without_entry_points(tmp_path, monkeypatch):
    names = [n for n in pi.EXPORTED if not n.startswith(("pi_cache", "pi_attn", "pi_matvec"))]
    said = load(tmp_path, monkeypatch, 5, names)
    assert "version 5" in said and "pi_matvec" in said


def test_the_same_version_without_an_entry_point(tmp_path, monkeypatch):
    said = load(tmp_path, monkeypatch, pi.ABI_VERSION, [n for n in pi.EXPORTED if n != "pi_attn_decode"])
    assert "pi_attn_decode" in said and "pi_attn_prompt" not in said


def test_another_version_with_all_of_them(tmp_path, monkeypatch):
    assert f"version {pi.ABI_VERSION + 1}" in load(tmp_path, monkeypatch, pi.ABI_VERSION + 1, pi.EXPORTED)


def test_a_library_that_says_no_version(tmp_path, monkeypatch):
    assert "None" in load(tmp_path, monkeypatch, 0, ["pi_status_str"])
