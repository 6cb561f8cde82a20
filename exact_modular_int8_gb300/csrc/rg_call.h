// rg_call.h -- host threads that share a workspace take turns (internal).
#pragma once

namespace rg {

// Held for the length of a call, its synchronisation included: what a call
// keeps in its workspace lives from its first launch to its last, and the status
// until it has been read, so no other call on that workspace may enqueue work in
// between.  Calls on different workspaces do not wait for each other.
class WorkspaceTurn {
 public:
  explicit WorkspaceTurn(const void* ws);
  ~WorkspaceTurn();
  WorkspaceTurn(const WorkspaceTurn&) = delete;
  WorkspaceTurn& operator=(const WorkspaceTurn&) = delete;

 private:
  const void* ws_;
};

}  // namespace rg
