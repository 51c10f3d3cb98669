// Calls that share a workspace launch one after the other.
#pragma once

#include <pthread.h>

namespace gemm_relu_hip {

// Held while a call with a workspace launches, by every entry point that takes one: the
// kernels of a call follow each other on their stream also when threads share the stream
// and with it the workspace, whose contents pass from one kernel to the next.  A thread
// sleeps while another's call with the same workspace launches; calls with other
// workspaces do not wait, also where that launch waits for room in its queue.  A turn is
// an entry on its thread's stack in the list of those held, so nothing is allocated.
class WorkspaceTurn {
    struct Turns {
        pthread_mutex_t mutex = PTHREAD_MUTEX_INITIALIZER;
        pthread_cond_t ended = PTHREAD_COND_INITIALIZER;
        WorkspaceTurn* held = nullptr;
    };
    static Turns& turns()
    {
        static Turns t;          // (constant initializers, nothing to destroy)
        return t;
    }

    const void* const workspace_;
    WorkspaceTurn* next_ = nullptr;

public:
    // NULL: a call that uses none.
    explicit WorkspaceTurn(const void* workspace) : workspace_(workspace)
    {
        if (!workspace_) return;
        Turns& t = turns();
        pthread_mutex_lock(&t.mutex);
        const auto taken = [&] {
            for (const WorkspaceTurn* h = t.held; h; h = h->next_)
                if (h->workspace_ == workspace_) return true;
            return false;
        };
        while (taken()) pthread_cond_wait(&t.ended, &t.mutex);
        next_ = t.held;
        t.held = this;
        pthread_mutex_unlock(&t.mutex);
    }
    WorkspaceTurn(const WorkspaceTurn&) = delete;
    WorkspaceTurn& operator=(const WorkspaceTurn&) = delete;
    ~WorkspaceTurn()
    {
        if (!workspace_) return;
        Turns& t = turns();
        pthread_mutex_lock(&t.mutex);
        if (t.held == this) {
            t.held = next_;
        } else {
            WorkspaceTurn* h = t.held;
            while (h->next_ != this) h = h->next_;
            h->next_ = next_;
        }
        pthread_cond_broadcast(&t.ended);
        pthread_mutex_unlock(&t.mutex);
    }
};

}  // namespace gemm_relu_hip
