// Ownership of the workspaces that a handle replaces by larger ones (host side).
#pragma once

#include <hip/hip_runtime.h>

#include <new>

namespace spense {

// A captured call records the addresses of the handle's workspaces, and its
// graph may be replayed for as long as the handle lives, also after a call that
// needed larger ones.  So a workspace that a captured call used is kept when it
// is replaced, and freed with the handle; the others are freed at once (a
// handle that only grows, one row at a time, then holds no more than it needs).
template <int N>
class GraphKept {
 public:
  GraphKept() = default;
  GraphKept(const GraphKept&) = delete;
  GraphKept& operator=(const GraphKept&) = delete;
  ~GraphKept() {
    while (kept_) {
      Node* n = kept_;
      kept_ = n->next;
      (void)hipFree(n->p);
      delete n;
    }
  }

  // A call on `s` is about to use the workspaces.
  void used(hipStream_t s) {
    if (all_ || !s) return;  // the null stream is never captured
    hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &st) != hipSuccess) (void)hipGetLastError();
    if (st == hipStreamCaptureStatusNone) return;
    for (bool& r : recorded_) r = true;
    all_ = true;
  }

  // Workspace i is being replaced: frees p, or keeps it if a graph may hold it.
  // False if it cannot be kept (no host memory); p is then still in use.
  bool drop(int i, void* p) {
    if (!p) return true;
    if (recorded_[i]) {
      Node* n = new (std::nothrow) Node{p, kept_};
      if (!n) return false;
      kept_ = n;
    } else {
      (void)hipFree(p);
    }
    recorded_[i] = all_ = false;
    return true;
  }

 private:
  struct Node {
    void* p;
    Node* next;
  };
  Node* kept_ = nullptr;
  bool recorded_[N] = {};
  bool all_ = false;  // every entry of recorded_
};

enum : int { kWsX = 0, kWsPartials = 1, kWsCounters = 2, kWorkspaces = 3 };

}  // namespace spense
